"""More of what the C calls of the layer norm, of the 8-bit form and of the
embedding refuse (not gpu): every refused call ends before any device work."""

import pytest

from test_rows_refusals import P, built, embedding_config, norm_config, refused  # noqa: F401 (built: a fixture)
from zero_sharded_mixed_flatparameter_gb300 import binding as B


@pytest.mark.parametrize("stride", [0, 1, 63])
def test_rows_of_an_output_that_overlap(stride):
    packed = B.zero_packed(P, P, 0)
    refused(B.zero_layer_norm, norm_config(), 4, P, 64, P, P, P, stride, P, packed)
    for x, kept in ((P, None), (0, packed)):
        refused(B.zero_layer_norm_backward, norm_config(), 4, P, 64, x, 64, kept, P, P, P, stride, P, P, 1, P, 1 << 40)
    refused(B.zero_unpack_activations, 4, 64, packed, P, 1, stride)
    cfg = embedding_config(dim=64)
    refused(B.zero_embedding, cfg, 4, P, P, 64, P, stride)
    for accumulate in (0, 1):
        refused(B.zero_embedding_backward, cfg, 4, P, P, 64, P, 1, stride, accumulate, P, 1 << 40)


@pytest.mark.parametrize("rows,most", [(1 << 30, 1 << 20), ((1 << 29) + 1, 1 << 20), (1 << 24, 1 << 26), ((1 << 20) + 1, 1 << 29)])
def test_a_sort_of_many_seconds(rows, most):
    cfg = embedding_config(rows=rows, dim=1)
    need = B.zero_embedding_backward_workspace_bytes(cfg, most)
    assert need >= 16 * most + 4 * rows
    refused(B.zero_embedding_backward_workspace_bytes, cfg, most + 1)
    refused(B.zero_embedding_backward, cfg, most + 1, P, P, 1, P, 1, 1, 0, P, 1 << 60)
    for fewer in (1, 1 << 17, 1 << 20):  # rows that a vocabulary has: any number of tokens
        B.zero_embedding_backward_workspace_bytes(embedding_config(rows=fewer, dim=1), 1 << 30)
