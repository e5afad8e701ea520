"""The feed-forward block's and the distillation's calls refuse pointers into the middle of an
element before anything is launched (no GPU needed)."""
import ctypes

import pytest

import sparse_top_lookup_gb300 as pk


@pytest.fixture(scope="module")
def L():
    if not __import__("os").path.exists(pk.LIB_PATH):
        pk.build()
    return pk.lib()


ARGS = dict(z=16, idx=16, t=16, loss=16, lse=16, dl=16, dz=16, st=16)


def forward(L, a):
    return L.pkm_distill(a["z"], pk.PKM_F32, 64, 4, 64, a["idx"], a["t"], 3, 1.0, a["loss"],
                         a["lse"], a["st"], None)


def backward(L, a):
    return L.pkm_distill_backward(a["z"], pk.PKM_F32, 64, 4, 64, a["idx"], a["t"], 3, 1.0, a["lse"],
                                  a["dl"], a["dz"], 64, a["st"], None)


def train(L, a):
    return L.pkm_distill_train(a["z"], pk.PKM_F32, 64, 4, 64, a["idx"], a["t"], 3, 1.0, a["dl"],
                               a["loss"], a["lse"], a["dz"], 64, a["st"], None)


@pytest.mark.parametrize("call,names", [(forward, "z idx t loss lse st"),
                                        (backward, "z idx t lse dl dz st"),
                                        (train, "z idx t loss lse dl dz st")])
def test_distill_refuses_parts_of_elements(L, call, names):
    for n in names.split():
        assert call(L, dict(ARGS, **{n: 18})) == pk.PKM_ERR_ALIGN, n
    assert call(L, dict(ARGS, idx=20)) == pk.PKM_ERR_ALIGN  # int64


def test_ffn_refuses_part_of_a_status_word(L):
    p = ctypes.c_void_p(16)
    assert L.pkm_gated_ffn(p, p, p, p, 4, 64, 64, 0, p, p, None, None, 18, None) == pk.PKM_ERR_ALIGN
    assert L.pkm_gated_ffn_backward(p, p, p, p, p, p, p, 4, 64, 64, 0, p, p, p, p, p, pk.PKM_BF16, 18,
                                    None) == pk.PKM_ERR_ALIGN
