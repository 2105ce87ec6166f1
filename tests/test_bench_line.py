"""The benchmark's line stands alone on stdout, short enough to be read whole from
the end of a log; the other configurations go to stderr (no GPU needed)."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_line_and_configurations_go_apart(capsys):
    line = {"metric": bench.METRIC, "value": 1.0, "clocks": {"sm_mhz": 1.0}}
    configs = [{"name": "c%d" % i, "text": "x" * 400} for i in range(40)]
    bench.emit(line, configs, {"samples": 3})
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and json.loads(out) == line
    assert err.count("\n") == 1 and json.loads(err) == {"configs": configs, "configs_clocks": {"samples": 3}}


def test_line_without_configurations(capsys):
    bench.emit({"value": 2.0})
    out, err = capsys.readouterr()
    assert json.loads(out) == {"value": 2.0} and err == ""
