"""What the calls around the decode step leave behind for the steps that follow: empty and
released slots, queries that are not finite, checkpoints, workspaces of captured calls.
Needs a B200; marked gpu."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import dynamic_sparse_attention_block_b200 as prr  # noqa: E402
from tests.test_gpu_serving import Case, _i32, _prompt, _shared, _some  # noqa: E402

DEV = "cuda"
NAN, INF = float("nan"), float("inf")


def _tokens(n, *heads, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(n, h, d, generator=g, device=DEV).bfloat16() for h in heads]


def _step(dec, mode, q, k=None, v=None):
    """One decode step; k, v: the token it appends ("host": appended by a call of its own before it)."""
    if mode == "fused":
        dec.step_fused(q, k_new=k, v_new=v)
    elif mode == "host":
        if k is not None:
            dec.append(k, v)
        dec.step_fused(q)
    else:
        if k is not None:
            dec.k_new.copy_(k)
            dec.v_new.copy_(v)
        dec.step(q, append=k is not None)
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- predictions

@pytest.mark.parametrize("mode", ["fused", "streams"])
@pytest.mark.parametrize("released", [False, True])
@pytest.mark.parametrize("n,P,cap", [(1, 8, 1024), (10, 64, 1024), (64, 2, 1024), (200, 7, 256), (900, 15, 1024)])
def test_a_prompt_shorter_than_the_prediction_in_an_empty_slot(n, P, cap, released, mode):
    """A fresh or released slot predicts as the zero state does at the length that its prompt gives it: the step
    equals that of a decoder that was prefilled, and reports nothing."""
    Hq, Hkv, d, bs = 8, 2, 64, 64
    sizes = dict(B=1, Hq=Hq, Hkv=Hkv, d=d, bs=bs, cap_tokens=cap, K=4, P=P)
    dec = prr.PRRDecoder(prr.Dims(pages=40, **sizes), empty=True)
    k, v, q = _tokens(n, Hkv, Hkv, Hq, d=d)
    if released:
        k0, v0, q0 = _tokens(250, Hkv, Hkv, Hq, d=d, seed=1)
        dec.reserve([251])
        dec.append_prompt(k0, v0, [0, 250])
        _step(dec, mode, q0[:1])
        dec.release([0])
    dec.reserve([n])
    dec.append_prompt(k, v, [0, n])
    flat = prr.PRRDecoder(prr.Dims(**sizes))
    flat.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    for x in (dec, flat):
        _step(x, mode, q[-1:])
    assert flat.device_status() == 0 and dec.device_status() == 0
    for name in ("sel", "missed", "n_missed", "keep", "pred"):
        a, b = getattr(dec, name), getattr(flat, name)
        if name == "missed":  # entries past the count are left as they were
            m = int(dec.n_missed.max())
            a, b = a[..., :m], b[..., :m]
        assert torch.equal(a, b), name
    assert (dec.out - flat.out).abs().max() < 1e-5 and (dec.lse - flat.lse).abs().max() < 1e-5


@pytest.mark.parametrize("entries", [[4, -1, -1], [0, 4, -1], [-2, -1, -1], [1, 0, -1], [0, 1, 3]])
def test_a_prediction_of_blocks_that_are_not_there_is_still_reported(entries):
    n, Hkv, Hq, d = 130, 1, 2, 64  # three blocks of a cache of sixteen
    dec = prr.PRRDecoder(prr.Dims(B=1, Hq=Hq, Hkv=Hkv, d=d, bs=64, cap_tokens=1024, K=2, P=3))
    k, v, q = _tokens(n, Hkv, Hkv, Hq, d=d)
    dec.prefill(k.transpose(0, 1)[None], v.transpose(0, 1)[None], n)
    dec.pred.copy_(_i32([[entries]]))
    _step(dec, "fused", q[-1:])
    assert dec.device_status() == 2
