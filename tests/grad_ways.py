"""Which way the library does a weight gradient (csrc/grad_plan.hpp), asked of its own rule, and sizes
that take each of them."""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))

# 16-bit types and FP32: (way, cut) -> sizes m, n, k.  cut: "whole" tiles alone, "cut" ones alone
# (along the tokens, then joined), "mixed": whole tiles and then the last ones cut.
SIZES = {
    "16": {("teams", "whole"): [(301, 311, 100), (901, 2100, 700)], ("teams", "cut"): [(1003, 311, 417)],
           ("small", "whole"): [(121, 300, 500), (70, 3700, 3601)], ("small", "cut"): [(301, 101, 100), (1500, 522, 99)],
           ("large", "whole"): [(101, 3476, 2953)], ("large", "cut"): [(3001, 522, 3587)],
           ("large", "mixed"): [(2101, 3987, 6075), (2080, 4001, 6016)]},
    "32": {("teams", "whole"): [(101, 311, 100), (77, 900, 1000)], ("teams", "cut"): [(601, 101, 100), (2049, 311, 417)],
           ("small", "whole"): [(101, 522, 3587), (70, 3700, 3601)], ("small", "cut"): [(301, 311, 100), (2049, 1366, 734)],
           ("large", "whole"): [(301, 2210, 2953)], ("large", "cut"): [(1003, 522, 3587), (1001, 1155, 1685)]},
}


def _lib():
    path = os.path.join(HERE, "hip", "libweight_grad_plan.so")
    if not os.path.exists(path):
        from compressed_adamw_state_amd import build
        build.build_plan_lib()
    return ctypes.CDLL(path)


def way_of(kind, m, n, k):
    """((way, cut), bytes of workspace) for kind "16" or "32" """
    out = (ctypes.c_int64 * 6)()
    i = ctypes.c_int64
    _lib().weight_grad_plan(2 if kind == "32" else 0, i(m), i(n), i(-(-k // 128) * 128), out)
    way, tn, tk, whole, splits, size = out
    cut = "whole" if whole == tn * tk else "cut" if whole == 0 else "mixed"
    assert (splits > 1) == (cut != "whole")
    return (("teams", "small", "large")[way], cut), size
