"""The prompts' C ABI and binding without a GPU: refusals on the host before
any HIP call."""
import pytest
import torch

import speculative_sampling_verify_spec_amd as sv

F32, BF16 = sv.SPECV_F32, sv.SPECV_BF16
BASE = 0x10000  # fake device addresses: every call fails before it could touch them


@pytest.fixture(scope="module")
def lib():
    return sv.load()


def attend(lib, **kw):
    a = dict(q=BASE, qs=0, k=2 * BASE, v=3 * BASE, ks=0, starts=4 * BASE, scale=0.1, B=4, T=100, H=8, Hq=32, D=128,
             out=5 * BASE, lse=None, dtype=BF16)
    a.update(kw)
    return lib.spec_prompt_attention(a["q"], a["qs"], a["k"], a["v"], a["ks"], a["starts"], a["scale"], a["B"], a["T"],
                                     a["H"], a["Hq"], a["D"], a["out"], a["lse"], a["dtype"], None)


PACKED = [
    (dict(dtype=2), -3), (dict(dtype=-1), -3), (dict(q=None), -1), (dict(k=None), -1), (dict(starts=None), -1),
    (dict(B=0), -2), (dict(B=65536), -2), (dict(T=0), -2), (dict(T=(1 << 24) + 1), -2), (dict(D=80), -2),
    (dict(D=0), -2), (dict(H=0), -2), (dict(H=1 << 15, Hq=1 << 15), -2), (dict(Hq=0), -2), (dict(Hq=12), -2),
    (dict(Hq=1 << 15), -2), (dict(Hq=8 * 1025), -2), (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2),
    (dict(scale=-3.2e38), -2), (dict(qs=100), -2), (dict(qs=-1), -2), (dict(qs=32 * 128 + 4), -6),
    (dict(ks=8 * 128 - 8), -2), (dict(qs=1 << 24), -2), (dict(ks=1 << 24), -2),  (dict(ks=8 * 128 + 1), -6), (dict(q=BASE + 2), -6), (dict(k=BASE + 8), -6),
    # rows of a sequence and workgroups of a grid are counted in 32 bits
    (dict(T=1 << 24, H=1, Hq=64), -2), (dict(T=1 << 24, H=128, Hq=128), -2), (dict(B=65535, T=1, H=256, Hq=256), -2)]


@pytest.mark.parametrize("kw,code", PACKED + [(dict(v=None), -1), (dict(out=None), -1), (dict(v=BASE + 8), -6),
                                              (dict(out=BASE + 8), -6)])
def test_attention_refusals(lib, kw, code):
    assert attend(lib, **kw) == code


def test_binding_refusals():
    x = torch.zeros(5, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        sv.prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int32))


def weigh(lib, **kw):
    a = dict(q=BASE, qs=0, k=2 * BASE, ks=0, lse=3 * BASE, starts=4 * BASE, scale=0.1, B=4, T=100, H=8, Hq=32, D=128,
             out=5 * BASE, C=100, dtype=BF16)
    a.update(kw)
    return lib.spec_prompt_weights(a["q"], a["qs"], a["k"], a["ks"], a["lse"], a["starts"], a["scale"], a["B"], a["T"],
                                   a["H"], a["Hq"], a["D"], a["out"], a["C"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", PACKED + [(dict(lse=None), -1), (dict(out=None), -1), (dict(C=0), -2),
                                              (dict(C=1 << 31), -2)])
def test_weights_refusals(lib, kw, code):
    assert weigh(lib, **kw) == code


def test_weights_binding_refuses_host_tensors():
    x = torch.zeros(5, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        sv.prompt_weights(x, x, torch.zeros(5, 4), torch.zeros(2, dtype=torch.int32), 5)


def test_row_strides():
    from speculative_sampling_verify_spec_amd._prompt import _row
    x = torch.zeros(5, 10, 64)
    assert _row("x", x[:, :4], 4, 64) == 640 and _row("x", x, 10, 64) == 640 and _row("x", x[:, 9:], 1, 64) == 640
    assert _row("x", x[:1, :4], 4, 64) == 256 and _row("x", x[:0, :4], 4, 64) == 256 and _row("x", x[::2], 10, 64) == 1280
    for bad in (x[:, ::2], x[..., ::2], x.transpose(1, 2), x[:1].expand(5, 10, 64), x[:, :1].expand(5, 10, 64)):
        with pytest.raises(ValueError):
            _row("x", bad, bad.shape[1], bad.shape[2])
