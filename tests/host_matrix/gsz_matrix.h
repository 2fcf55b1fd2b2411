// For the CPU run: gsz_device.h beside this file holds these, too.
#pragma once
#include "gsz_device.h"
