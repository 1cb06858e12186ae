"""The last build's AdamW and gradient kernels (no GPU): recorded, and with
the waves in flight that their streams need (figures as in
tests/test_build_cpu.py)."""
from test_build_cpu import _rows


def test_list_kernels_keep_their_occupancy():
    rows = {r["kernel"]: int(r["occupancy"]) for r in _rows()}
    want = {"adamw_kernelILi32E": 6, "adamw_kernelILi8E": 6, "adamw_read_kernel": 8, "grad_sumsq_kernel": 8,
            "grad_scale_kernel": 8, "grad_norm_finish_kernel": 1, "grad_norm_small_kernel": 1}
    for name, waves in want.items():
        found = [o for k, o in rows.items() if name in k]
        assert found and min(found) >= waves, (name, found)
