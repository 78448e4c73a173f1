"""What the C calls of the layer norm, of the 8-bit form and of the embedding
refuse (not gpu): every call here ends before any device work."""

import pytest

from zero_sharded_mixed_flatparameter_gb300 import binding as B

P = 1 << 20  # an address that no check can tell from a real one


@pytest.fixture(scope="module", autouse=True)
def built():
    from zero_sharded_mixed_flatparameter_gb300 import build_lib
    build_lib.build()
    B.load()


def refused(call, *args):
    with pytest.raises(B.ZeroError) as e:
        call(*args)
    assert e.value.status == B.ZERO_EINVAL
    assert B.zero_last_error(None)


def norm_config(**over):
    base = dict(cols=64, center=1, dtype=1, weight_dtype=1, eps=1e-5)
    base.update(over)
    return B.zero_norm_config(*base.values())


@pytest.mark.parametrize("over", [
    dict(cols=0), dict(cols=-1), dict(cols=(1 << 24) + 1), dict(center=2), dict(dtype=2), dict(dtype=-1),
    dict(weight_dtype=3), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=-1), dict(x=0),
    dict(x=P + 2), dict(y=0), dict(y=P + 2), dict(x_stride=-1), dict(y_stride=-1), dict(weight=P + 2), dict(bias=P + 2),
    dict(stats=P + 4), dict(codes=0), dict(codes=P + 8), dict(scales=0), dict(format=2), dict(format=-1)], ids=str)
def test_layer_norm(over):
    o = dict(rows=4, x=P, y=P, x_stride=64, y_stride=64, weight=P, bias=P, stats=P, codes=P, scales=P, format=0)
    cfg = norm_config(**{k: v for k, v in over.items() if k in dict(B.zero_norm_config._fields_)})
    o.update({k: v for k, v in over.items() if k in o})
    refused(B.zero_layer_norm, cfg, o["rows"], o["x"], o["x_stride"], o["weight"], o["bias"], o["y"], o["y_stride"],
            o["stats"], B.zero_packed(o["codes"], o["scales"], o["format"]))


@pytest.mark.parametrize("over", [
    dict(cols=0), dict(center=-1), dict(dtype=2), dict(rows=-1), dict(dy=0), dict(dy=P + 2), dict(x=0), dict(x=P + 2),
    dict(dx=0), dict(dx=P + 1), dict(dy_stride=-1), dict(x_stride=-1), dict(dx_stride=-1), dict(weight=P + 2),
    dict(stats=0), dict(stats=P + 4), dict(dweight=P + 2), dict(dbias=P + 2), dict(dgrad_dtype=2), dict(workspace=0),
    dict(workspace=P + 8), dict(packed=B.zero_packed(0, P, 0)), dict(packed=B.zero_packed(P, 0, 0)),
    dict(packed=B.zero_packed(P, P, 7)), dict(packed=B.zero_packed(P + 1, P, 0))], ids=str)
def test_layer_norm_backward(over):
    o = dict(rows=4, dy=P, dy_stride=64, x=P, x_stride=64, packed=None, weight=P, stats=P, dx=P, dx_stride=64, dweight=P,
             dbias=P, dgrad_dtype=1, workspace=P, workspace_bytes=1 << 40)
    cfg = norm_config(**{k: v for k, v in over.items() if k in dict(B.zero_norm_config._fields_)})
    o.update({k: v for k, v in over.items() if k in o})
    refused(B.zero_layer_norm_backward, cfg, *o.values())


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(cols=0), dict(cols=(1 << 24) + 1), dict(dtype=2), dict(x=0), dict(x=P + 2), dict(stride=-1),
    dict(packed=B.zero_packed(0, P, 0)), dict(packed=B.zero_packed(P + 4, P, 0)), dict(packed=B.zero_packed(P, 0, 1)),
    dict(packed=B.zero_packed(P, P, 2)), dict(packed=None)], ids=str)
def test_pack(over):
    o = dict(rows=4, cols=64, x=P, dtype=1, stride=64, packed=B.zero_packed(P, P, 0))
    o.update(over)
    refused(B.zero_pack_activations, *o.values())
    refused(B.zero_unpack_activations, o["rows"], o["cols"], o["packed"], o["x"], o["dtype"], o["stride"])


def embedding_config(**over):
    base = dict(rows=10, dim=16, dtype=1, id_bytes=8, scale=1.0)
    base.update(over)
    return B.zero_embedding_config(*base.values())


CONFIGS = [dict(rows=-1), dict(rows=(1 << 30) + 1), dict(dim=0), dict(dim=(1 << 24) + 1), dict(dtype=2), dict(id_bytes=2),
           dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=-1), dict(tokens=(1 << 30) + 1)]


@pytest.mark.parametrize("over", CONFIGS + [
    dict(ids=0), dict(ids=P + 4), dict(table=0), dict(table=P + 2), dict(table_stride=-1), dict(out=0), dict(out=P + 2),
    dict(out_stride=-1)], ids=str)
def test_embedding(over):
    o = dict(tokens=4, ids=P, table=P, table_stride=16, out=P, out_stride=16)
    cfg = embedding_config(**{k: v for k, v in over.items() if k in dict(B.zero_embedding_config._fields_)})
    o.update({k: v for k, v in over.items() if k in o})
    refused(B.zero_embedding, cfg, *o.values())


@pytest.mark.parametrize("over", CONFIGS + [
    dict(ids=0), dict(ids=P + 4), dict(dout=0), dict(dout=P + 2), dict(dout_stride=-1), dict(dtable=0), dict(dtable=P + 2),
    dict(dtable_dtype=2), dict(dtable_stride=-1), dict(accumulate=2), dict(workspace=0), dict(workspace=P + 8),
    dict(workspace_bytes=95)], ids=str)
def test_embedding_backward(over):
    o = dict(tokens=4, ids=P, dout=P, dout_stride=16, dtable=P, dtable_dtype=1, dtable_stride=16, accumulate=0,
             workspace=P, workspace_bytes=1 << 40)
    cfg = embedding_config(**{k: v for k, v in over.items() if k in dict(B.zero_embedding_config._fields_)})
    o.update({k: v for k, v in over.items() if k in o})
    refused(B.zero_embedding_backward, cfg, *o.values())


def test_no_work():
    # nothing to do: no pointer is looked at, nothing is launched
    B.zero_layer_norm(norm_config(), 0, 0, 0, 0, 0, 0, 0, 0)
    B.zero_pack_activations(0, 5, 0, 0, 0, B.zero_packed(0, 0, 0))
    B.zero_unpack_activations(0, 5, B.zero_packed(0, 0, 0), 0, 0, 0)
    B.zero_embedding(embedding_config(), 0, 0, 0, 0, 0, 0)
    B.zero_embedding_backward(embedding_config(rows=0), 5, 0, 0, 0, 0, 1, 0, 0, 0, 0)
    B.zero_embedding_backward(embedding_config(), 0, 0, 0, 0, 0, 1, 0, 1, 0, 0)
    B.zero_layer_norm_backward(norm_config(), 0, 0, 0, 0, 0, None, 0, 0, 0, 0, 0, 0, 1, 0, 0)


def test_workspaces_grow_with_the_work():
    sizes = [B.zero_embedding_backward_workspace_bytes(embedding_config(), t) for t in (0, 1, 32, 33, 1000, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    runs = (1 << 20) // 32
    assert sizes[-1] >= 8 * (1 << 20) + 4 * 11 + 4 * runs + runs * 2 * 16 * 4
    for cfg in (embedding_config(dim=0), embedding_config(rows=-1)):
        refused(B.zero_embedding_backward_workspace_bytes, cfg, 4)
    refused(B.zero_layer_norm_backward_workspace_bytes, norm_config(cols=0), 4)
    refused(B.zero_layer_norm_backward_workspace_bytes, norm_config(), -1)
