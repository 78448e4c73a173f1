"""Muon steps and orthogonalisations through the products' split and paired
forms and through several batches against the index-checking debug build (not
collected by pytest: tests/test_gpu_muon_debug_products.py runs this file in a
subprocess, so that this process loads the debug library)."""

import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

from zero_sharded_mixed_flatparameter_gb300 import binding as B, build_lib  # noqa: E402

B.load(build_lib.build(debug_checks=True))

import torch  # noqa: E402

from muon_reference import NS_TOL, orthogonalized64, relative  # noqa: E402
from test_gpu_muon import check_matrices, grads_for, make, reduced, snapshot, step  # noqa: E402
from test_gpu_muon_products import MANY, params  # noqa: E402
from zero_sharded_mixed_flatparameter_gb300 import ops  # noqa: E402
from zero_sharded_mixed_flatparameter_gb300.runner import FlatStep  # noqa: E402


def main():
    for name, mats in MANY.items():
        pl, shapes = params(mats)
        fs = make(pl, shapes, 2)
        grads = grads_for(fs, pl, 2, "bf16", 1)
        before = snapshot(fs)
        step(fs, grads)
        check_matrices(fs, pl, shapes, before, reduced(grads))
        fs.close()
    for batch, rows, cols in ((1, 512, 2048), (1, 1024, 1024), (4, 512, 2048), (2, 2048, 2100)):
        x = torch.randn(batch, rows, cols, device="cuda")
        got = ops.orthogonalize(x)
        assert relative(got[0], orthogonalized64(x[0])) <= NS_TOL
    assert B.zero_debug_check_failures() == 0, B.zero_debug_check_failures()
    print("no check failed", flush=True)
    for rows, cols in ((1024, 1024), (2048, 2100)):  # a split and a paired matrix at the end of the buffer
        fs = FlatStep([rows * cols], [0], stage=0, n_ranks=1, init_params=[torch.randn(rows * cols).cuda()])
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
