"""Muon steps against the index-checking debug build of the library (not
collected by pytest: tests/test_gpu_muon_debug.py runs this file in a
subprocess, so that this process loads the debug library).

First no check may fail and the results must be the ones of the formulas; then
the kernels are told that the arrays end 8 elements early (they do not, so no
access can leave them) and must leave those elements alone."""

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

from zero_sharded_mixed_flatparameter_gb300 import binding as B, build_lib  # noqa: E402

B.load(build_lib.build(debug_checks=True))

import torch  # noqa: E402

from test_gpu_muon import check_matrices, grads_for, make, mlp, reduced, snapshot, step  # noqa: E402


def main():
    for widths, n in (([13, 57, 131, 9], 3), ([300, 700, 130], 8), ([40, 1500, 24], 2), ([260, 260, 260], 4)):
        pl, shapes = mlp(widths)
        fs = make(pl, shapes, n)
        for t in range(2):
            grads = grads_for(fs, pl, n, "bf16", t + 1)
            before = snapshot(fs)
            step(fs, grads)
            check_matrices(fs, pl, shapes, before, reduced(grads))
        fs.close()
    assert B.zero_debug_check_failures() == 0, B.zero_debug_check_failures()
    print("no check failed", flush=True)
    for sizes in ([64, 96], [150, 200]):  # a thin and a larger matrix at the end of the buffer
        rows, cols = sizes
        init = [torch.randn(rows * cols).cuda()]
        from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep
        fs = FlatStep([rows * cols], [0], stage=0, n_ranks=1, init_params=init)
        fs.enable_muon([(rows, cols)], lr=0.1)
        before, failed = fs.master.clone(), B.zero_debug_check_failures()
        B.zero_debug_inject(fs.ctx, B.ZERO_INJECT_SHORT_BOUNDS)
        fs.reduce_grads(-1, [torch.randn(rows * cols).bfloat16().cuda()])
        fs.step()
        fs.post_step()
        torch.cuda.synchronize()
        assert B.zero_debug_check_failures() > failed
        assert torch.equal(fs.master[-8:], before[-8:]) and not torch.equal(fs.master[:-8], before[:-8])
        fs.close()
    print("short bounds refused: ok", flush=True)


if __name__ == "__main__":
    main()
