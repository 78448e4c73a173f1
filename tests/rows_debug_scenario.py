"""Layer norm, 8-bit form and embedding against the index-checking debug build of
the library (not collected by pytest: tests/test_gpu_rows_debug.py runs this file
in a subprocess, so that this process loads the debug library).

The sorted tokens and the list of rows in parts are indexes that one launch
writes and another follows: no check of them may fail, and the results must be
the ones of the formulas."""

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

from zero_sharded_mixed_flatparameter_gb300 import binding as B, build_lib  # noqa: E402

B.load(build_lib.build(debug_checks=True))

import torch  # noqa: E402

import test_gpu_rows_batches as batches  # noqa: E402
from rows_reference import E4M3, INT8  # noqa: E402


def main():
    for tokens, rows, dim, kind in ((20011, 400, 2048, "any"), (12007, 300, 2047, "any"), (40009, 70000, 263, "text"),
                                    (20011, 3, 2048, "one"), (25013, 5, 1536, "text"), (700, 260000, 8, "any"), (1, 1, 1, "one")):
        for dtype in (torch.float32, torch.bfloat16):
            batches.test_embedding_gradient(tokens, rows, dim, kind, dtype, torch.bfloat16)
    for rows, cols in ((38011, 264), (5003, 1301), (1603, 8192), (70001, 40)):
        batches.test_layer_norm(rows, cols, True, torch.bfloat16)
    for form in (E4M3, INT8):
        batches.test_pack(9001, 777, torch.float32, form)
    assert B.zero_debug_check_failures() == 0, B.zero_debug_check_failures()
    print("no check failed: ok", flush=True)


if __name__ == "__main__":
    main()
