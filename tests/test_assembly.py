"""Assembly statements say which registers they change."""
import pathlib
import re

SOURCES = [p for p in (pathlib.Path(__file__).parent.parent / "gradient_sync_zero_amd").rglob("*") if p.suffix in (".h", ".hip", ".cpp")]


def statements():
    for p in SOURCES:
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", p.read_text(), re.S):
            yield p.name, m.group(1)


def test_m0_is_named_where_it_is_written():
    found = [(name, s) for name, s in statements() if re.search(r"\bs_\w+\s+m0\s*,", s)]
    assert found                                         # the loads to LDS
    for name, s in found:
        changed = s.rsplit(":", 1)[1]
        assert '"m0"' in changed, (name, s)
