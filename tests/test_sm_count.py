"""Launches size themselves by the SMs that the device reports: no count of them stands in the code.  Host code only."""

import re

from test_dependent_launches import _all_sources


def test_no_count_of_sms_is_written_down():
    for name, text in _all_sources().items():
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
        assert not re.search(r"\b152\b", code), name
