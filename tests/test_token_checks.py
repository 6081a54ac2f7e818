"""CPU-only: block norms, convolution, recurrence and log probabilities refuse
what they do not take, before anything reaches the GPU (fake aligned addresses,
never dereferenced) -- and the torch helpers refuse wrong types, shapes and
devices."""
import ctypes
import os
import re

import pytest
import torch

from quant_dequant_gemv_amd import binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH),
                                reason="libqkgemv.so not built (run __graft_entry__.build())")

M = 1 << 28  # fake regions M apart
TYPE, SHAPE, PTR, FLAGS, OK = b.QK_EINVAL_TYPE, b.QK_EINVAL_SHAPE, b.QK_EINVAL_PTR, b.QK_EINVAL_FLAGS, b.QK_OK
INF, NAN = float("inf"), float("nan")


def heads(at, row=512, head=128, elem=1, f16=0):
    return b.qk_heads(at * M, row, head, elem, f16)


# ------------------------------------------------------------------ block norm

def block(**kw):
    return b.qk_block(*{**dict(post_norm=10 * M, pre_norm=11 * M, eps=1e-6, scale=1.0, act=1), **kw}.values())


def norm(blk=None, rows=4, groups=4, dim=128, y=heads(1), gate=None, res=None, h=None, x=heads(2)):
    return b.qk_block_norm(blk or block(), rows, groups, dim, y, gate, res, h, x)


def test_block_norm_arguments():
    for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(groups=0), dict(groups=4097), dict(dim=0), dict(dim=32769),
               dict(rows=1 << 22, groups=9), dict(blk=block(eps=-1.0)), dict(blk=block(eps=NAN)), dict(blk=block(eps=INF)),
               dict(blk=block(scale=NAN)), dict(blk=block(scale=-INF)), dict(y=heads(1, row=-1)), dict(x=heads(2, row=100)),
               dict(x=heads(2, elem=0))):
        assert norm(**kw) == SHAPE, kw
    for act in (-1, 3):
        assert norm(block(act=act)) == FLAGS
    assert b.qk_block_norm(None, 4, 4, 128, heads(1), None, None, None, heads(2)) == PTR
    for kw in (dict(y=None), dict(x=None), dict(y=heads(0)), dict(x=b.qk_heads(2 * M + 2, 512, 128, 1, 0)),
               dict(blk=block(post_norm=10 * M + 2)), dict(blk=block(pre_norm=11 * M + 1))):
        assert norm(**kw) == PTR, kw
    assert norm(y=heads(1, f16=2)) == TYPE and norm(gate=heads(3, f16=-1)) == TYPE
    assert norm(rows=0) == OK


def test_block_norm_overlaps():
    for x in (b.qk_heads(M + 4, 512, 128, 1, 0), heads(1, f16=1), heads(3), heads(10), heads(11)):
        # over its input shifted, over it in another type, over the residual in another layout, over the weights
        assert norm(x=x, res=heads(3, row=1024)) == PTR
    assert norm(h=heads(2), x=heads(2)) == PTR  # h and x are two outputs
    assert norm(h=heads(5), x=b.qk_heads(5 * M + 8, 512, 128, 1, 0)) == PTR
    assert norm(gate=heads(3), x=b.qk_heads(3 * M - 4, 512, 128, 1, 0)) == PTR


# ------------------------------------------------------------------ sequences with a state

def seqs(**kw):
    a = dict(rows=4, nseq=2, q_start=20 * M, slots=21 * M, slots_out=22 * M, kv_len=23 * M, commit=24 * M)
    return b.qk_state_seqs(*{**a, **kw}.values())


def conv(**kw):
    a = dict(pool=10 * M, num_slots=8, channels=256, taps=4, weight=11 * M, bias=12 * M)
    return b.qk_conv(*{**a, **kw}.values())


def delta(**kw):
    return b.qk_delta(*{**dict(pool=10 * M, num_slots=8, k_heads=2, v_heads=4, key_dim=128, value_dim=64), **kw}.values())


def rows(**kw):
    a = dict(q=heads(1, 256), k=heads(2, 256), v=heads(3, 256, 64), alpha=heads(4, 4, 1, 0), beta=heads(5, 4, 1, 0), A=13 * M,
             dt_bias=14 * M, eps=1e-6, scale=0.1, norm=1)
    return b.qk_delta_rows(*{**a, **kw}.values())


X, Y = heads(1, 256, 0), heads(2, 256, 0)
OUT = heads(6, 256, 64)
WS = (30 * M, 1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 22) + 1), SHAPE), (dict(nseq=0), SHAPE), (dict(nseq=65537), SHAPE),
    (dict(q_start=None, rows=5), SHAPE), (dict(slots=None), PTR), (dict(slots=21 * M + 2), PTR), (dict(q_start=20 * M + 1), PTR),
    (dict(slots_out=22 * M + 2), PTR), (dict(kv_len=23 * M + 3), PTR), (dict(commit=24 * M + 2), PTR),
])
def test_every_call_checks_its_sequences(kw, code):
    assert b.qk_conv_silu(conv(), seqs(**kw), 1, X, Y) == code
    assert b.qk_delta_rule(delta(), seqs(**kw), rows(), OUT, *WS) == code
    if code == SHAPE:
        assert b.qk_delta_workspace_bytes(delta(), seqs(**kw)) == -1


def test_conv_arguments():
    for kw in (dict(num_slots=0), dict(num_slots=1 << 31), dict(channels=0), dict(channels=65537), dict(taps=1), dict(taps=9)):
        assert b.qk_conv_silu(conv(**kw), seqs(), 1, X, Y) == SHAPE
    for kw in (dict(pool=None), dict(pool=10 * M + 8), dict(weight=None), dict(weight=11 * M + 2), dict(bias=12 * M + 1)):
        assert b.qk_conv_silu(conv(**kw), seqs(), 1, X, Y) == PTR
    for act in (-1, 2, 3):
        assert b.qk_conv_silu(conv(), seqs(), act, X, Y) == FLAGS
    assert b.qk_conv_silu(None, seqs(), 1, X, Y) == PTR and b.qk_conv_silu(conv(), None, 1, X, Y) == PTR
    assert b.qk_conv_silu(conv(), seqs(), 1, None, Y) == PTR
    assert b.qk_conv_silu(conv(), seqs(), 1, heads(1, f16=3), Y) == TYPE
    assert b.qk_conv_silu(conv(), seqs(), 1, X, heads(2, 255, 0)) == SHAPE
    assert b.qk_conv_silu(conv(), seqs(rows=0), 1, X, Y) == OK
    for at in (1, 10, 11, 12, 20, 21, 22, 23, 24):  # y over x, the state, the weights, the tables
        assert b.qk_conv_silu(conv(), seqs(), 1, X, heads(at, 256, 0)) == PTR
    assert b.qk_conv_silu(conv(pool=1 * M), seqs(), 1, X, Y) == PTR
    assert b.qk_conv_silu(conv(), seqs(slots=10 * M + 4), 1, X, None) == PTR


def test_delta_arguments():
    for kw in (dict(num_slots=0), dict(num_slots=1 << 31), dict(k_heads=0), dict(v_heads=0), dict(v_heads=5), dict(v_heads=4098),
               dict(k_heads=4097, v_heads=4097), dict(key_dim=96), dict(key_dim=256), dict(value_dim=0), dict(value_dim=48),
               dict(value_dim=544)):
        assert b.qk_delta_rule(delta(**kw), seqs(), rows(), OUT, *WS) == SHAPE, kw
        assert b.qk_delta_workspace_bytes(delta(**kw), seqs()) == -1
    for kw in (dict(eps=-1.0), dict(eps=NAN), dict(scale=INF), dict(scale=NAN)):
        assert b.qk_delta_rule(delta(), seqs(), rows(**kw), OUT, *WS) == SHAPE
    assert b.qk_delta_rule(delta(), seqs(), rows(norm=2), OUT, *WS) == FLAGS
    for kw in (dict(A=13 * M + 2), dict(dt_bias=14 * M + 1), dict(A=None), dict(q=heads(0)), dict(alpha=b.qk_heads(4 * M + 2, 4, 1, 0, 0))):
        assert b.qk_delta_rule(delta(), seqs(), rows(**kw), OUT, *WS) == PTR, kw
    assert b.qk_delta_rule(delta(), seqs(), rows(beta=heads(5, f16=2)), OUT, *WS) == TYPE
    assert b.qk_delta_rule(delta(pool=None), seqs(), rows(), OUT, *WS) == PTR
    assert b.qk_delta_rule(delta(pool=10 * M + 4), seqs(), rows(), OUT, *WS) == PTR
    assert b.qk_delta_rule(None, seqs(), rows(), OUT, *WS) == PTR and b.qk_delta_rule(delta(), None, rows(), OUT, *WS) == PTR
    assert b.qk_delta_rule(delta(), seqs(), None, OUT, *WS) == PTR
    assert b.qk_delta_rule(delta(), seqs(rows=0), rows(), OUT, None, 0) == OK
    assert b.qk_delta_workspace_bytes(delta(), seqs(rows=0)) == 0
    for at in (1, 2, 3, 4, 5, 10, 13, 14, 20, 21, 22, 23, 24):
        assert b.qk_delta_rule(delta(), seqs(), rows(), heads(at, 256, 64), *WS) == PTR, at
    assert b.qk_delta_rule(delta(pool=3 * M), seqs(), rows(), OUT, *WS) == PTR
    assert b.qk_delta_rule(delta(), seqs(), rows(), heads(6, 256, 63), *WS) == SHAPE
    # 2^27 columns of states pass, more do not
    one = seqs(rows=65536, nseq=65536, q_start=None)
    for hv, ok in ((32, True), (33, False)):
        assert (b.qk_delta_workspace_bytes(delta(k_heads=1, v_heads=hv), one) >= 0) == ok


def test_delta_workspace():
    long = seqs(rows=4096, nseq=1, q_start=None)
    need = b.qk_delta_workspace_bytes(delta(), long)
    assert need >= 0
    if need:
        assert b.qk_delta_rule(delta(), long, rows(), OUT, 30 * M, need - 1) == SHAPE
        for ws in (None, 30 * M + 8, 1 * M, 3 * M, 6 * M, 10 * M, 21 * M):
            assert b.qk_delta_rule(delta(), long, rows(), OUT, ws, need) == PTR


# ------------------------------------------------------------------ log probabilities

def probs(**kw):
    a = dict(tokens=10 * M, token_lp=11 * M, lse=12 * M, entropy=13 * M, top_ids=14 * M, top_lp=15 * M, ntok=2, top=5)
    return b.qk_probs(*{**a, **kw}.values())


def test_logprobs_arguments():
    z = heads(1, 70000, 0)
    call = lambda z=z, rows=4, vocab=70000, scale=1.0, o=probs(), ws=WS: b.qk_logprobs(z, rows, vocab, scale, o, *ws)  # noqa: E731
    for kw in (dict(rows=-1), dict(rows=(1 << 22) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(vocab=1 << 40),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(scale=2.0 ** 65), dict(o=probs(top=65)),
               dict(o=probs(top=-1)), dict(o=probs(ntok=-1)), dict(o=probs(ntok=1025)), dict(z=heads(1, -1))):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(z=None), dict(z=heads(0)), dict(o=None), dict(o=probs(tokens=None)), dict(o=probs(token_lp=None)),
               dict(o=probs(ntok=0)), dict(o=probs(top=0)), dict(o=probs(top_ids=None)), dict(o=probs(top_lp=None)),
               dict(o=b.qk_probs()), dict(o=probs(lse=12 * M + 2)), dict(o=probs(tokens=10 * M + 1)), dict(o=probs(lse=1 * M)),
               dict(o=probs(entropy=10 * M)), dict(o=probs(entropy=12 * M + 4)), dict(o=probs(top_lp=14 * M + 8))):
        assert call(**kw) == PTR, kw
    assert call(z=heads(1, 70000, 0, f16=5)) == TYPE
    assert call(rows=0, ws=(None, 0)) == OK
    need = b.qk_logprobs_workspace_bytes(z, 4, 70000, 5)
    assert need > 0  # a few rows are cut into parts
    assert call(ws=(30 * M, need - 1)) == SHAPE
    for ws in (None, 30 * M + 8, 1 * M, 10 * M, 15 * M):
        assert call(ws=(ws, need)) == PTR
    assert b.qk_logprobs_workspace_bytes(z, 4, 0, 5) == b.qk_logprobs_workspace_bytes(z, 4, 10, 65) == -1


# ------------------------------------------------------------------ the torch helpers

def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


I32 = torch.int32


def test_helpers_refuse():
    y, w, slots = z(4, 2, 64), z(64), z(2, dtype=I32)
    c = b.ConvState(3, z(64, 4), z(64))
    d = b.DeltaState(3, 1, 2, 64, 64, pool=z(3, 2, 64, 64))
    q, v, al = z(4, 1, 64), z(4, 2, 64), z(4, 2)
    assert tuple(c.pool.shape) == (3, 3, 64)
    for exc, match, call in (
        (TypeError, "float16", lambda: b.block_norm(y.double())),
        (TypeError, "tensor", lambda: b.block_norm(None)),
        (ValueError, "shape", lambda: b.block_norm(z(4, 64))),
        (ValueError, "act", lambda: b.block_norm(y, gate=y, act="relu")),
        (ValueError, "pre_norm", lambda: b.block_norm(y, pre_norm=z(63))),
        (TypeError, "post_norm", lambda: b.block_norm(y, post_norm=w.half())),
        (TypeError, "weight", lambda: b.ConvState(3, z(64, 4).half())),
        (ValueError, "weight", lambda: b.ConvState(3, z(64))),
        (ValueError, "bias", lambda: b.ConvState(3, z(64, 4), z(63))),
        (ValueError, "pool", lambda: b.ConvState(3, z(64, 4), pool=z(3, 4, 64))),
        (b.QKError, None, lambda: b.ConvState(3, z(64, 9))),
        (b.QKError, None, lambda: b.ConvState(0, z(64, 4))),
        (b.QKError, None, lambda: b.DeltaState(3, 2, 3, 64, 64)),
        (b.QKError, None, lambda: b.DeltaState(3, 1, 2, 80, 64)),
        (b.QKError, None, lambda: b.DeltaState(3, 1 + 2 ** 32, 2, 64, 64)),
        (ValueError, "pool", lambda: b.DeltaState(3, 1, 2, 64, 64, pool=z(3, 2, 64, 32))),
        (TypeError, "pool", lambda: b.DeltaState(3, 1, 2, 64, 64, pool=z(3, 2, 64, 64).half())),
        (ValueError, "shape", lambda: b.conv_silu(c, z(4, 63), slots)),
        (TypeError, "float16", lambda: b.conv_silu(c, z(4, 64).long(), slots)),
        (TypeError, "int32", lambda: b.conv_silu(c, z(4, 64), slots.long())),
        (ValueError, "q_start", lambda: b.conv_silu(c, z(4, 64), slots, q_start=slots)),
        (ValueError, "commit", lambda: b.conv_silu(c, z(4, 64), slots, commit=z(3, dtype=I32))),
        (ValueError, "act", lambda: b.conv_silu(c, z(4, 64), slots, act="sigmoid")),
        (ValueError, "shape", lambda: b.delta_rule(d, z(4, 2, 64), q, v, al, al, slots)),
        (ValueError, "shape", lambda: b.delta_rule(d, q, q, z(5, 2, 64), al, al, slots)),
        (ValueError, "alpha", lambda: b.delta_rule(d, q, q, v, z(4, 3), al, slots)),
        (ValueError, "A ", lambda: b.delta_rule(d, q, q, v, al, al, slots, A=z(3))),
        (ValueError, "without A", lambda: b.delta_rule(d, q, q, v, al, al, slots, dt_bias=z(2))),
        (ValueError, "contiguous", lambda: b.delta_rule(d, q, q, v, al, al, z(4, dtype=I32)[::2])),
        (ValueError, "shape", lambda: b.logprobs(z(4))),
        (TypeError, "int32", lambda: b.logprobs(z(4, 9), z(4, 1))),
        (ValueError, "tokens", lambda: b.logprobs(z(4, 9), z(3, 1, dtype=I32))),
        (b.QKError, None, lambda: b.logprobs(z(4, 9), top=65)),
        # sizes right, tensors on the host
        (ValueError, "CUDA", lambda: b.block_norm(y, w, y, residual=y, pre_norm=w)),
        (ValueError, "CUDA", lambda: b.conv_silu(c, z(4, 64), slots)),
        (ValueError, "CUDA", lambda: b.delta_rule(d, q, q, v, al, al, slots)),
        (ValueError, "CUDA", lambda: b.logprobs(z(4, 9), top=3)),
    ):
        with pytest.raises(exc, match=match):
            call()


def test_struct_layouts_match_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qkgemv.h")).read()
    for name, size in (("qk_block", 32), ("qk_state_seqs", 48), ("qk_conv", 40), ("qk_delta", 32), ("qk_delta_rows", 232),
                       ("qk_probs", 56)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.strip(" *") for line in re.findall(r"([^;]+);", body) for f in line.strip().split(" ", 1)[1].replace("int32_t", "").split(",")]
        fields = [re.sub(r"^(float|int|void|char) ", "", f).strip(" *") for f in fields]
        assert fields == [f for f, _ in getattr(b, name)._fields_], name
        assert ctypes.sizeof(getattr(b, name)) == size, name


def test_states_keep_their_tensors():
    c = b.ConvState(3, z(64, 4), z(64))
    d = b.DeltaState(3, 1, 2, 64, 64, pool=z(3, 2, 64, 64))
    for o, name in ((c, "pool"), (c, "weight"), (c, "bias"), (d, "pool")):
        t = getattr(o, name)
        with pytest.raises(AttributeError):
            setattr(o, name, t.clone())
        assert getattr(o, name) is t
        t.fill_(1)
