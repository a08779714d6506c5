"""When bench.py's clock reading takes the driver's metrics table to have been
refreshed, with amdsmi and the GPU replaced by stand-ins (no GPU needed)."""
import os
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def reading(monkeypatch, tables):
    """The clock reading over a sequence of tables (the last one stays), and how many were read."""
    taken = []

    def metrics(handle):
        taken.append(tables[min(len(taken), len(tables) - 1)])
        return taken[-1]

    smi = types.ModuleType("amdsmi")
    smi.amdsmi_init = smi.amdsmi_shut_down = lambda: None
    smi.amdsmi_get_gpu_metrics_info = metrics
    monkeypatch.setitem(sys.modules, "amdsmi", smi)
    monkeypatch.setattr(bench, "_smi_handle", lambda amdsmi, torch: 0)
    event = types.SimpleNamespace(record=lambda stream: None, synchronize=lambda: None)
    cuda = types.SimpleNamespace(current_stream=lambda: None, Event=lambda: event, synchronize=lambda: None)
    return bench.clock_under_load(types.SimpleNamespace(cuda=cuda), None, [], [], "BF16X9", max_s=0.2), len(taken)


def table(counter, stamp, mhz, busy=100):
    t = {"firmware_timestamp": stamp, "current_gfxclks": [mhz, mhz], "current_socket_power": 1000, "average_gfx_activity": busy}
    return t if counter is None else {"accumulation_counter": counter, **t}


def test_the_counter_tells_refreshes_where_there_is_one(monkeypatch):
    """A time stamp that moves with every reading is no new interval: the
    reading is the one after the counter's second step."""
    tables = [table(5, 0, 500), *(table(5, i, 600) for i in (1, 2, 3)), *(table(6, i, 700) for i in (4, 5, 6)), table(7, 7, 800)]
    clock, _ = reading(monkeypatch, tables)
    assert clock is not None and clock["sclk_ghz"] == 0.8


@pytest.mark.parametrize("counter", [None, "N/A"])
def test_the_time_stamp_tells_them_where_there_is_none(monkeypatch, counter):
    tables = [table(counter, 0, 500), table(counter, 0, 500), table(counter, 1, 700), table(counter, 1, 700), table(counter, 2, 800)]
    clock, taken = reading(monkeypatch, tables)
    assert clock is not None and clock["sclk_ghz"] == 0.8 and taken == 5


def test_no_busy_interval(monkeypatch):
    clock, _ = reading(monkeypatch, [table(i, i, 500, busy=10) for i in range(4)])
    assert clock is None
