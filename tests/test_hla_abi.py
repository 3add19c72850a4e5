"""The C ABI of linear attention with one decay per head and of rotary positions refuses bad arguments on the host
(none of these calls reaches a CUDA API)."""
import pytest

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def K():
    from linear_attention_recurrence_11_b200 import build
    build.build()
    from linear_attention_recurrence_11_b200 import kda
    return kda


FWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, S0=None, o=FAKE, S_T=None, B=1, T=64, H=2, dk=128, dv=128, scale=1.0, dtype=1,
           gate=0, cu=None, num_seqs=0, ws=None, ws_bytes=0, status=None, stream=None, path=0)
BWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, S0=None, dO=FAKE, dS_T=None, dq=FAKE, dk_out=FAKE, dv_out=FAKE, dg=None, dS0=None,
           B=1, T=64, H=2, dk=128, dv=128, scale=1.0, dtype=1, gate=0, cu=None, num_seqs=0, ws=None, ws_bytes=0, status=None,
           stream=None, path=0)
DEC = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, S=FAKE, o=FAKE, N=2, H=2, dk=64, dv=64, scale=1.0, dtype=1, gate=0, stream=None)
ROPE = dict(q=FAKE, k=FAKE, pos=None, pos64=0, inv=FAKE, qo=FAKE, ko=FAKE, B=1, T=4, Hq=2, Hk=2, d=64, rot=64, inter=0,
            inverse=0, mscale=1.0, dtype=1, stream=None)


def caller(f, defaults):
    return lambda **kw: f(*{**defaults, **kw}.values())


@pytest.mark.parametrize("name,args", [("kda_hla_forward", FWD), ("kda_hla_backward", BWD)])
def test_prefill_refusals(K, name, args):
    f = caller(getattr(K._lib, name), args)
    for bad in (dict(B=0), dict(T=-1), dict(H=0), dict(dtype=2), dict(gate=2), dict(path=3), dict(path=9),
                dict(cu=FAKE, num_seqs=0), dict(cu=FAKE, num_seqs=2, B=2), dict(q=None), dict(k=None), dict(v=None), dict(g=None)):
        assert f(**bad) == K.KDA_ERR_INVALID_ARG, bad
    for bad in (dict(dk=48), dict(dv=256), dict(H=1 << 30, B=4), dict(path=2, dtype=0), dict(B=1 << 15, T=1 << 16)):
        assert f(**bad) == K.KDA_ERR_UNSUPPORTED, bad
    for n in ("q", "k", "v", "g", "S0", "ws", "status"):
        assert f(**{n: FAKE + 8}) == K.KDA_ERR_ALIGNMENT, n
    assert f() == K.KDA_ERR_WORKSPACE
    assert f(ws=FAKE, ws_bytes=128) == K.KDA_ERR_WORKSPACE


def test_backward_only_refusals(K):
    f = caller(K._lib.kda_hla_backward, BWD)
    for bad in (dict(dO=None), dict(dq=None), dict(dk_out=None), dict(dv_out=None), dict(gate=1, dg=FAKE)):
        assert f(**bad) == K.KDA_ERR_INVALID_ARG, bad
    for n in ("dO", "dS_T", "dq", "dk_out", "dv_out", "dg", "dS0"):
        assert f(**{n: FAKE + 4}) == K.KDA_ERR_ALIGNMENT, n


def test_decode_refusals(K):
    f = caller(K._lib.kda_hla_decode_step, DEC)
    for bad in (dict(N=0), dict(H=-1), dict(dtype=5), dict(gate=-1), dict(S=None), dict(o=None)):
        assert f(**bad) == K.KDA_ERR_INVALID_ARG, bad
    assert f(dk=16) == K.KDA_ERR_UNSUPPORTED
    assert f(S=FAKE + 4) == K.KDA_ERR_ALIGNMENT


def test_rope_refusals(K):
    f = caller(K._lib.kda_rope, ROPE)
    for bad in (dict(B=0), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(dtype=3), dict(rot=0), dict(rot=66), dict(rot=7), dict(q=None),
                dict(k=None), dict(Hk=0), dict(k=None, ko=None), dict(ko=None), dict(inv=None), dict(qo=None)):
        assert f(**bad) == K.KDA_ERR_INVALID_ARG, bad
    for bad in (dict(d=65, rot=64), dict(d=1026), dict(Hq=1 << 20), dict(B=1 << 20, T=1 << 20)):
        assert f(**bad) == K.KDA_ERR_UNSUPPORTED, bad
    for n in ("q", "k", "pos", "inv", "qo", "ko"):
        assert f(**{n: FAKE + 2}) == K.KDA_ERR_ALIGNMENT, n


def test_workspace_queries(K):
    import torch
    assert K.kda_hla_forward_workspace_size(1, 64, 2, 32, 64, 0, torch.float32) > 0
    assert K.kda_hla_backward_workspace_size(1, 100, 2, 128, 128, 3, torch.bfloat16) > 0
    assert K.kda_hla_forward_workspace_size(3, 0, 2, 32, 64, 0, torch.float32) == 0
    for bad in (dict(B=0), dict(dk=40), dict(num_seqs=-1), dict(B=2, num_seqs=2)):
        a = {**dict(B=1, T=64, H=2, dk=64, dv=64, num_seqs=0), **bad}
        with pytest.raises(K.KdaError):
            K.kda_hla_forward_workspace_size(*a.values(), torch.float32)
        with pytest.raises(K.KdaError):
            K.kda_hla_backward_workspace_size(*a.values(), torch.float32)
