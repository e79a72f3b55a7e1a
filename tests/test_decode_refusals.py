"""What the entry points between the linear layers refuse, on the host, before anything is launched."""
import ctypes

import pytest
import torch

from gemv_w4a16_gemm_gb300 import w4q

FAKE = 1 << 20   # a 16-byte aligned non-null "device" address, never dereferenced


def cache(**changes):
    c = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, seq_lens=FAKE, blocks=8, seqs=2, width=4,
             kv_heads=2, head_dim=128, page=64, format=0)
    c.update(changes)
    return ctypes.byref(w4q._Kv8Cache(*[c[n] for n, _ in w4q._Kv8Cache._fields_]))


def norm(**changes):
    a = dict(q=FAKE, k=FAKE, tokens=3, q_heads=4, k_heads=2, head_dim=128, q_stride=1024, k_stride=1024, q_weight=FAKE,
             k_weight=FAKE, eps=1e-6, cos_sin=FAKE, positions=10, rot=128, interleaved=0, pos=FAKE, q_out=FAKE,
             k_out=FAKE, stream=None)
    a.update(changes)
    return w4q.lib().qk_norm_rope(*a.values())


def append(c=None, **changes):
    a = dict(k=FAKE, v=FAKE, k_stride=1024, v_stride=1024, tokens=2, cu=None, q=FAKE, q_stride=1024, q_heads=4,
             q_out=FAKE, q_weight=None, k_weight=None, eps=1e-6, cos_sin=FAKE, positions=10, rot=64, interleaved=0,
             stream=None)
    a.update(changes)
    return w4q.lib().kv8_append(cache() if c is None else c, *a.values())


def attend(c=None, **changes):
    a = dict(q=FAKE, q_stride=1024, out=FAKE, lse=None, queries=1, heads=8, scale=0.1, window=0, workspace=None, bytes=0,
             stream=None)
    a.update(changes)
    return w4q.lib().kv8_attention(cache() if c is None else c, *a.values())


@pytest.mark.parametrize("changes,status", [
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(tokens=-1), 1), (dict(q_heads=0), 1), (dict(k=None), 1),
    (dict(k_out=None), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(positions=0), 1), (dict(rot=0), 1),
    (dict(q_stride=511), 1), (dict(k_stride=128), 1),
    (dict(head_dim=96), 2), (dict(rot=24), 2), (dict(rot=144), 2), (dict(tokens=1 << 30), 2), (dict(q_heads=2000, q_stride=1 << 20), 2),
    (dict(q=FAKE + 2), 3), (dict(k_out=FAKE + 8), 3), (dict(q_stride=1020), 3), (dict(cos_sin=FAKE + 4), 3), (dict(pos=FAKE + 4), 3),
    (dict(tokens=0), 0),
])
def test_norm_rope(changes, status):
    assert norm(**changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(k=None), 1), (dict(seq_lens=None), 1), (dict(blocks=0), 1), (dict(seqs=0), 1), (dict(width=-1), 1), (dict(kv_heads=0), 1),
    (dict(head_dim=80), 2), (dict(page=48), 2), (dict(page=8), 2), (dict(page=256), 2), (dict(format=2), 2), (dict(seqs=5000), 2),
    (dict(width=1 << 25), 2), (dict(blocks=1 << 31), 2),
    (dict(v=FAKE + 8), 3), (dict(k_scale=FAKE + 4), 3), (dict(block_table=FAKE + 4), 3),
])
def test_cache(changes, status):
    tokens = changes.get("seqs", 2)
    assert append(cache(**changes), tokens=tokens if 0 < tokens <= 4096 else 2) == status
    assert attend(cache(**changes)) == status
    assert w4q.lib().kv8_read(cache(**changes), None, 2, FAKE, FAKE, None) == status


def test_no_cache():
    assert append(ctypes.POINTER(w4q._Kv8Cache)()) == 1


@pytest.mark.parametrize("changes,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(tokens=3), 1), (dict(tokens=-1, cu=FAKE), 1), (dict(q=None), 1), (dict(q_out=None), 1),
    (dict(q_heads=-1), 1), (dict(k_stride=255), 1), (dict(v_stride=0), 1),
    (dict(rot=40), 2), (dict(tokens=1 << 30, cu=FAKE), 2),
    (dict(v=FAKE + 2), 3), (dict(k_stride=1028), 3), (dict(cu=FAKE + 4), 3), (dict(q_weight=FAKE + 2), 3),
    (dict(tokens=0, cu=FAKE), 0),
])
def test_append(changes, status):
    assert append(**changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(queries=0), 1), (dict(heads=0), 1), (dict(window=-1), 1), (dict(scale=float("nan")), 1),
    (dict(q_stride=1000), 1),
    (dict(heads=7), 2), (dict(queries=17), 2), (dict(heads=256, q_stride=1 << 15), 2),
    (dict(q=FAKE + 2), 3), (dict(out=FAKE + 2), 3), (dict(lse=FAKE + 4), 3), (dict(workspace=FAKE + 8), 3),
])
def test_attention(changes, status):
    assert attend(**changes) == status


def test_attention_over_too_many_positions():
    assert attend(cache(seqs=4096, width=1 << 20)) == 2


@pytest.mark.parametrize("args", [(0, 1, 8, 2, 128), (5000, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 7, 2, 128), (1, 65, 2, 2, 128),
                                  (1, 1, 8, 2, 96), (1, 1, 0, 2, 64)])
def test_workspace_of_unsupported_sizes(args):
    assert w4q.kv8_workspace_bytes(*args) == 0


def test_python_checks():
    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4q.qk_norm_rope(t)                     # not on the GPU
    with pytest.raises(ValueError):
        w4q.kv8_append(t, t, t, t, t, t, t, t)


@pytest.mark.gpu
def test_refused_calls_write_nothing(cuda):
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.int8, device=cuda)
    ks = torch.zeros(4, 2, device=cuda)
    table = torch.zeros(2, 2, dtype=torch.int32, device=cuda)
    lens = torch.tensor([3, 5], dtype=torch.int32, device=cuda)
    args = (kc, kc.clone(), ks, ks.clone(), table, lens)
    q = torch.ones(2, 1, 4, 64, dtype=torch.bfloat16, device=cuda)
    out = torch.full_like(q, 7.0)
    with pytest.raises(w4q.W4QError) as e:
        w4q.kv8_attention(q, *args, out=out, workspace=torch.zeros(64, dtype=torch.uint8, device=cuda))
    assert e.value.status == 4
    with pytest.raises(w4q.W4QError):
        w4q.kv8_attention(q, *args, out=out, window=-1)
    with pytest.raises(ValueError):
        w4q.kv8_attention(q.float(), *args, out=out)
    with pytest.raises(ValueError):
        w4q.kv8_attention(q[..., ::2], *args)
    with pytest.raises(ValueError):
        w4q.kv8_append(q[:, 0], q[:, 0], *args)          # 4 heads, the cache has 2
    with pytest.raises(ValueError):
        w4q.kv8_append(q[:, 0, :2], q[:1, 0, :2], *args)
    with pytest.raises(ValueError):
        w4q.kv8_read(*args, cu_tokens=table[0])
    with pytest.raises(ValueError):
        w4q.qk_norm_rope(q[:, 0].transpose(0, 1))
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (kc == 0).all()


def moe(**changes):
    a = dict(x=FAKE, router=FAKE, bias=None, w13=FAKE, w2=FAKE, out=FAKE, tokens=4, hidden=512, inter=256, experts=8, topk=2,
             sigmoid=0, renormalize=1, scale=1.0, ids=None, weights=None, workspace=None, bytes=0, stream=None)
    a.update(changes)
    return w4q.lib().moe_w4a16(*a.values())


@pytest.mark.parametrize("changes,status", [
    (dict(x=None), 1), (dict(w2=None), 1), (dict(out=None), 1), (dict(tokens=0), 1), (dict(topk=0), 1), (dict(topk=9), 1),
    (dict(inter=-256), 1), (dict(bias=FAKE), 1), (dict(scale=float("nan")), 1),
    (dict(tokens=65), 2), (dict(hidden=300), 2), (dict(inter=128), 2), (dict(experts=513), 2), (dict(experts=40, topk=17), 2),
    (dict(hidden=1 << 16), 2),
    (dict(x=FAKE + 2), 3), (dict(w13=FAKE + 8), 3), (dict(ids=FAKE + 4), 3), (dict(workspace=FAKE + 4), 3),
    (dict(), 4), (dict(workspace=FAKE, bytes=100), 4),
])
def test_moe(changes, status):
    assert moe(**changes) == status


def test_moe_workspace():
    assert w4q.moe_workspace_bytes(4, 512, 256, 8, 2) > 4 * 512 * 2
    assert w4q.moe_workspace_bytes(65, 512, 256, 8, 2) == 0
    assert w4q.moe_workspace_bytes(4, 512, 100, 8, 2) == 0
