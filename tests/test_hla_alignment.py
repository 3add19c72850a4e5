"""Addresses that the C ABI of linear attention and of rotary positions refuses on the host: what is read by element may begin at
any element, but not inside one (none of these calls reaches a CUDA API)."""
import pytest

from test_hla_abi import BWD, DEC, FAKE, FWD, K, ROPE, caller  # noqa: F401


@pytest.mark.parametrize("name,args", [("kda_hla_forward", FWD), ("kda_hla_backward", BWD)])
def test_offsets(K, name, args):  # noqa: F811
    f = caller(getattr(K._lib, name), args)
    assert f(cu=FAKE + 2, num_seqs=2) == K.KDA_ERR_ALIGNMENT
    for at in (4, 8, 12):  # (goes on to the workspace)
        assert f(cu=FAKE + at, num_seqs=2) == K.KDA_ERR_WORKSPACE


def test_gates_of_a_decode_step(K):  # noqa: F811
    f = caller(K._lib.kda_hla_decode_step, DEC)
    for bad in (dict(g=FAKE + 1), dict(dtype=0, g=FAKE + 2), dict(gate=1, g=FAKE + 2)):
        assert f(**bad) == K.KDA_ERR_ALIGNMENT, bad


def test_positions_and_frequencies(K):  # noqa: F811
    f = caller(K._lib.kda_rope, ROPE)
    for bad in (dict(pos=FAKE + 2), dict(pos=FAKE + 4, pos64=1), dict(inv=FAKE + 2)):
        assert f(**bad) == K.KDA_ERR_ALIGNMENT, bad


def test_rows_of_rotary_positions(K):  # noqa: F811
    f = caller(K._lib.kda_rope, ROPE)
    for n in ("q", "k", "qo", "ko"):
        for bad in (dict(d=64, at=8), dict(d=64, dtype=0, at=8), dict(d=60, at=4), dict(d=58, at=2), dict(d=58, dtype=0, at=4)):
            kw = {i: j for i, j in bad.items() if i != "at"}
            assert f(rot=2, **{n: FAKE + bad["at"]}, **kw) == K.KDA_ERR_ALIGNMENT, (n, bad)
