"""What the drafted-round calls refuse, checked before anything is launched: the C
entries' status codes and the binding's exceptions, on a host without a GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_86_gb300 as pkv
from paged_kv_cache_86_gb300 import _lib
from paged_kv_cache_86_gb300.build import build

BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32
ARG, SHAPE, DTYPE, WORKSPACE = -1, -2, -3, -4
A, B, C = 256, 4096, 8192        # aligned addresses that are never followed


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


# ------------------------------------------------------------ C entry points --

def rope(lib, **kw):
    a = dict(q_out=A, qos=1024, k_out=B, kos=256, q=C, k=C, qs=1536, ks=1536, qw=None, kw=None,
             eps=1e-6, pos=A, table=A, maxp=100, r=128, inter=0, t=3, hq=8, hkv=2, d=128, dtype=0)
    a.update(kw)
    return lib.pkv_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=1), DTYPE), (dict(t=-1), ARG), (dict(hq=0), ARG), (dict(hkv=0), ARG),
    (dict(maxp=0), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(d=96), SHAPE), (dict(r=0), SHAPE), (dict(r=24), SHAPE), (dict(r=144), SHAPE),
    (dict(q_out=None), ARG), (dict(k_out=None), ARG), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(pos=None), ARG), (dict(table=None), ARG), (dict(table=260), ARG), (dict(q=264), ARG),
    (dict(qw=264), ARG), (dict(kw=264), ARG), (dict(qs=1023), ARG), (dict(qs=1028), ARG),
    (dict(ks=255), ARG), (dict(qos=8), ARG), (dict(kos=8), ARG), (dict(kos=260), ARG),
    (dict(q_out=C), ARG),        # in place at another stride
    (dict(k_out=C), ARG),
    (dict(t=0), 0), (dict(t=0, q=None), 0),
])
def test_norm_rope_status(lib, change, status):
    assert rope(lib, **change) == status


def store(lib, **kw):
    a = dict(q_out=A, qos=1024, q=C, k=C, v=C, qs=1536, ks=1536, vs=1536, qw=None, kw=None,
             eps=1e-6, pos=A, table=A, maxp=100, r=128, inter=0, kc=A, vc=A, slots=A, t=3, hq=8,
             hkv=2, d=128, bs=16, nb=4, dtype=0)
    a.update(kw)
    return lib.pkv_qk_norm_rope_store(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), DTYPE), (dict(bs=0), ARG), (dict(nb=0), ARG), (dict(v=None), ARG),
    (dict(kc=None), ARG), (dict(vc=None), ARG), (dict(slots=None), ARG), (dict(v=264), ARG),
    (dict(vs=128), ARG), (dict(vs=260), ARG), (dict(d=80), SHAPE), (dict(r=8), SHAPE),
    (dict(q=None), ARG), (dict(t=0), 0),
])
def test_norm_rope_store_status(lib, change, status):
    assert store(lib, **change) == status


def plan(lib, **kw):
    a = dict(ctx=A, new=B, s=2, bt=A, mb=4, free=A, nf=9, cur=A, cur_out=B, slots=A, pos=A, mt=8,
             cq=A, ck=A, out=C, bs=16, nb=4)
    a.update(kw)
    return lib.pkv_plan_slots(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(s=-1), dict(mb=-1), dict(nf=-1), dict(mt=-1), dict(bs=0), dict(nb=0), dict(cur=None),
    dict(cur_out=None), dict(cq=None), dict(ck=None), dict(ctx=None), dict(new=None),
    dict(out=None), dict(bt=None), dict(slots=None), dict(pos=None), dict(free=None),
    dict(cur_out=A), dict(out=A), dict(out=B), dict(nb=1 << 27), dict(mb=1 << 27),
])
def test_plan_refusals(lib, change):
    assert plan(lib, **change) == ARG


def masks(lib, **kw):
    a = dict(par=A, cu=A, ctx=A, s=2, total=8, mq=8, mask=A, words=1, pos=A)
    a.update(kw)
    return lib.pkv_tree_masks(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(s=-1), ARG), (dict(total=-1), ARG), (dict(mq=-1), ARG), (dict(mq=33), ARG),
    (dict(mq=65535 * 128 + 1, words=1 << 20), ARG), (dict(par=None), ARG), (dict(cu=None), ARG),
    (dict(ctx=None), ARG), (dict(mask=None), ARG), (dict(pos=None), ARG),
    (dict(s=0), 0), (dict(total=0), 0), (dict(mq=0), 0),
])
def test_masks_status(lib, change, status):
    assert masks(lib, **change) == status


@pytest.mark.parametrize("out,name", [("mask", "par"), ("mask", "cu"), ("mask", "ctx"), ("pos", "par"),
                                      ("pos", "cu"), ("pos", "ctx"), ("pos", "mask")])
def test_masks_outputs_over_inputs(lib, out, name):
    """CTAs read what others would be writing."""
    at = dict(par=A, cu=A + 4096, ctx=A + 8192, mask=A + 12288, pos=A + 16384)
    at[out] = at[name]
    assert masks(lib, **at) == ARG


def tree(lib, **kw):
    a = dict(out=A, q=A, key=A, value=A, ks=1536, vs=1536, kc=A, vc=A, bt=A, mb=4, ctx=A, cu=A,
             mask=A, words=1, s=2, total=8, mq=8, mc=64, hq=8, hkv=2, d=128, bs=16, nb=4,
             scale=0.1, ws=A, wb=1 << 30, dtype=0)
    a.update(kw)
    return lib.pkv_tree_decode(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), DTYPE), (dict(s=-1), ARG), (dict(total=-1), ARG), (dict(mq=-1), ARG),
    (dict(mc=-1), ARG), (dict(hq=0), ARG), (dict(hkv=0), ARG), (dict(bs=0), ARG), (dict(nb=0), ARG),
    (dict(mb=-1), ARG), (dict(scale=float("inf")), ARG), (dict(scale=3e38), ARG),
    (dict(d=64), SHAPE), (dict(hq=9), SHAPE), (dict(hq=34), SHAPE), (dict(mc=65), ARG),
    (dict(mq=33), ARG), (dict(nb=1 << 27), ARG), (dict(out=None), ARG), (dict(q=None), ARG),
    (dict(key=None), ARG), (dict(value=None), ARG), (dict(kc=None), ARG), (dict(vc=None), ARG),
    (dict(bt=None), ARG), (dict(ctx=None), ARG), (dict(cu=None), ARG), (dict(mask=None), ARG),
    (dict(out=264), ARG), (dict(q=264), ARG), (dict(key=264), ARG), (dict(value=264), ARG),
    (dict(ks=248), ARG), (dict(ks=260), ARG), (dict(vs=248), ARG), (dict(ws=None), WORKSPACE),
    (dict(ws=128), WORKSPACE), (dict(wb=16), WORKSPACE),
    (dict(s=0), 0), (dict(total=0), 0), (dict(mq=0), 0),
])
def test_tree_status(lib, change, status):
    assert tree(lib, **change) == status


def test_tree_workspace_of_refused_shapes(lib):
    assert pkv.tree_decode_workspace_size(8, 9, 2) == 0
    assert pkv.tree_decode_workspace_size(8, 34, 2) == 0
    assert pkv.tree_decode_workspace_size(8, 8, 2, 64) == 0
    assert pkv.tree_decode_workspace_size(-1, 8, 2) == 0


# ------------------------------------------------------------------- binding --

def rope_args():
    return dict(q=torch.zeros(3, 8, 128, dtype=BF16), k=torch.zeros(3, 2, 128, dtype=BF16),
                positions=torch.zeros(3, dtype=I32), cos_sin=torch.zeros(9, 128, dtype=F32))


def store_args():
    a = rope_args()
    a.update(v=torch.zeros(3, 2, 128, dtype=BF16), k_cache=torch.zeros(4, 16, 2, 128, dtype=BF16),
             v_cache=torch.zeros(4, 16, 2, 128, dtype=BF16), slot_mapping=torch.zeros(3, dtype=I32))
    return a


def plan_args():
    return dict(context_lens=torch.zeros(2, dtype=I32), new_lens=torch.zeros(2, dtype=I32),
                block_tables=torch.zeros(2, 4, dtype=I32), free_blocks=torch.zeros(9, dtype=I32),
                free_cursor=torch.zeros(1, dtype=I32), block_size=16, num_blocks=8, max_tokens=5)


def masks_args():
    return dict(parents=torch.zeros(6, dtype=I32), cu_seqlens_q=torch.zeros(3, dtype=I32),
                context_lens=torch.zeros(2, dtype=I32), max_seqlen_q=4)


def tree_args():
    return dict(q=torch.zeros(6, 8, 128, dtype=BF16), key=torch.zeros(6, 2, 128, dtype=BF16),
                value=torch.zeros(6, 2, 128, dtype=BF16),
                k_cache=torch.zeros(4, 16, 2, 128, dtype=BF16),
                v_cache=torch.zeros(4, 16, 2, 128, dtype=BF16),
                block_tables=torch.zeros(2, 4, dtype=I32), context_lens=torch.zeros(2, dtype=I32),
                cu_seqlens_q=torch.zeros(3, dtype=I32), tree_mask=torch.zeros(6, 1, dtype=I32),
                scale=0.1, max_seqlen_q=4)


CALLS = {"rope": (pkv.qk_norm_rope, rope_args), "store": (pkv.qk_norm_rope_store, store_args),
         "plan": (pkv.plan_slots, plan_args), "masks": (pkv.tree_masks, masks_args),
         "tree": (pkv.tree_decode, tree_args)}


@pytest.mark.parametrize("call", CALLS)
def test_dense_host_tensors_pass_the_layout_and_fail_the_device(call):
    f, args = CALLS[call]
    with pytest.raises(TypeError, match="CUDA tensor"):
        f(**args())


def tensors_of(call):
    return [n for n, v in CALLS[call][1]().items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in tensors_of(c)])
def test_wrong_type_rank_or_layout(call, name):
    f, args = CALLS[call]
    a = args()
    t = a[name]
    a[name] = t.to(torch.float16 if t.is_floating_point() else torch.int64)
    with pytest.raises(TypeError, match=name):
        f(**a)
    a[name] = t.unsqueeze(0)
    with pytest.raises(ValueError, match=name):
        f(**a)
    a[name] = t.tolist()
    with pytest.raises(TypeError, match=name):
        f(**a)
    # the last dim at twice its stride
    a[name] = torch.zeros(*t.shape[:-1], 2 * t.shape[-1] + 2, dtype=t.dtype)[..., ::2][..., :t.shape[-1]]
    if t.shape[-1] > 1:
        with pytest.raises(ValueError, match=name):
            f(**a)


@pytest.mark.parametrize("call,name", [("rope", "positions"), ("rope", "k"), ("store", "slot_mapping"),
                                       ("store", "v"), ("store", "k_cache"), ("plan", "new_lens"),
                                       ("plan", "context_lens"), ("masks", "context_lens"),
                                       ("masks", "cu_seqlens_q"), ("tree", "key"), ("tree", "value"),
                                       ("tree", "block_tables"), ("tree", "cu_seqlens_q"),
                                       ("tree", "tree_mask"), ("tree", "v_cache")])
def test_sizes_that_do_not_match(call, name):
    f, args = CALLS[call]
    a = args()
    a[name] = torch.cat([a[name], a[name][:1]])
    with pytest.raises(ValueError):
        f(**a)


def test_weights_outputs_and_counts():
    a = rope_args()
    with pytest.raises(ValueError, match="q_weight must have head_dim"):
        pkv.qk_norm_rope(**a, q_weight=torch.zeros(64, dtype=BF16))
    with pytest.raises(TypeError, match="k_weight"):
        pkv.qk_norm_rope(**a, k_weight=torch.zeros(128, dtype=F32))
    with pytest.raises(ValueError, match="q_out"):
        pkv.qk_norm_rope(**a, q_out=torch.zeros(3, 4, 128, dtype=BF16))
    with pytest.raises(ValueError, match="k_out rows"):
        pkv.qk_norm_rope(**a, k_out=torch.zeros(3, 128, 2, dtype=BF16).transpose(1, 2))
    with pytest.raises(ValueError, match="max_tokens"):
        pkv.plan_slots(**{**plan_args(), "max_tokens": -1})
    with pytest.raises(ValueError, match="one cursor"):
        pkv.plan_slots(**{**plan_args(), "free_cursor": torch.zeros(2, dtype=I32)})
    buf = [torch.zeros(n, dtype=I32) for n in (5, 5, 3, 3, 2, 2)]
    with pytest.raises(ValueError, match="out.free_cursor must have 1"):
        pkv.plan_slots(**plan_args(), out=pkv.SlotPlan(*buf))
    with pytest.raises(ValueError, match="tree_mask must have one row"):
        pkv.tree_masks(**masks_args(), tree_mask=torch.zeros(5, 1, dtype=I32))
    with pytest.raises(ValueError, match="positions must have one entry"):
        pkv.tree_masks(**masks_args(), positions=torch.zeros(5, dtype=I32))
