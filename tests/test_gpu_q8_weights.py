"""The 8-bit decode's probabilities: one heavy key in front of a long tail of light ones, values with a mean, so
that what the digits of the weights drop does not average out.

The weights of a tile of 128 tokens are digits against the tile's own largest weight, w (times V scale). E4M3:
two digits, each weight off by at most 2^-9 of itself, or 2^-22 w where it is below the digits' normal range.
int8: three digits, a step of w / (32512 * 128), off by at most half of it, 2^-23 w rounded up to 2^-22. With
A = sum P |V| and the largest |V| of the sequence, all tokens of all tiles together move an output by at most
2^-9 A + 128 * 2^-22 max|V| or 128 * 2^-22 max|V| (the tiles' largest weights add up to at most 1). Scores of up
to 32 (log2 units) carry three fp32 roundings, 2^-17 together, and each exponential and sum rounds a few more
times: 2^-14 A covers them. The output's own rounding to bf16 is half a step, 2^-8 of it."""

import math

import pytest
import torch

import attention_online_softmax_fwd_b200 as ab

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def values(codes):
    return codes.view(E4M3).double() if codes.dtype == torch.uint8 else codes.double()


def codes_of(x, kind):
    return x.to(E4M3).view(torch.uint8) if kind == "e4m3" else torch.round(x).clamp(-127, 127).to(torch.int8)


def reference(q, k, v, lens):
    """float64: o, log-sum-exp and sum P |V| of every row; k, v [tokens, Hkv, D] shared by all sequences."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros(N, Hq, D, dtype=torch.float64, device=q.device)
    a, lse = torch.zeros_like(o), torch.zeros(N, Hq, dtype=torch.float64, device=q.device)
    for b, L in enumerate(lens):
        for h in range(k.shape[1]):
            s = q[b, h * G:(h + 1) * G].double() @ k[:L, h].T / math.sqrt(D)
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            p = torch.softmax(s, -1)
            o[b, h * G:(h + 1) * G], a[b, h * G:(h + 1) * G] = p @ v[:L, h], p @ v[:L, h].abs()
    return o, lse, a


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 8, 128), (8, 4, 128), (32, 8, 128), (10, 2, 128), (16, 2, 128), (32, 2, 128),
                                      (8, 8, 64), (24, 6, 64), (16, 2, 64), (32, 2, 64)])
@pytest.mark.parametrize("spread", [0.0, 0.6])
def test_heavy_key_before_a_long_tail(cuda_device, kind, Hq, Hkv, D, spread):
    """Score gaps of 6 to 20 nats between key 0, whose value is zero, and the rest, whose values have a mean of 1;
    from one tile to 313, some sequences cut and most of them not."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(7100 + Hq + Hkv + D)
    T, page, block = 40000, 64, 16
    u = torch.randint(0, 2, (Hkv, D), generator=g, device=dev) * 2.0 - 1
    k = torch.randn(T, Hkv, D, generator=g, device=dev) * spread
    k[0] = u
    v = 1.0 + 0.25 * torch.randn(T, Hkv, D, generator=g, device=dev)
    v[0] = 0.0
    step = 2.0 ** -5
    kc, vc = codes_of(k / step, kind), codes_of(v / step, kind)
    kc, vc = [t.view(T // page, page, Hkv, D).contiguous() for t in (kc, vc)]
    ks = torch.full((T // page, page // block, Hkv), step, device=dev)
    vs = ks.clone()
    lens = [60, 128, 129, 1000, 8192, 8200, 40000] * 4
    N = len(lens)
    gap = 6.0 + 14.0 * torch.rand(N, Hq, generator=g, device=dev)
    q = gap[..., None] / math.sqrt(D) * u.repeat_interleave(Hq // Hkv, 0)
    q = q.to(torch.bfloat16)
    bt = torch.arange(T // page, dtype=torch.int32, device=dev).expand(N, -1).contiguous()
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)
    o, lse = ab.decode_paged_q8(q, kc, vc, ks, vs, bt, sl)
    kk, vv = values(kc).view(T, Hkv, D) * step, values(vc).view(T, Hkv, D) * step
    ref, l_ref, a = reference(q, kk, vv, lens)
    own = (2.0 ** -9 if kind == "e4m3" else 0.0) + 2.0 ** -14
    bound = 2.0 ** -8 * ref.abs() + own * a + 2.0 ** -15 * vv.abs().max()
    err = (o.double() - ref).abs()
    worst = (err / bound).flatten(1).amax(1)
    print(kind, (Hq, Hkv, D), "error / bound by length", [f"{n}: {float(worst[i::7].max()):.2f}" for i, n in enumerate(lens[:7])],
          "max", float(err.max()))
    assert (err <= bound).all()
    assert (lse.double() - l_ref).abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
def test_value_scale_far_above_its_neighbours(cuda_device, kind, D):
    """One block of 16 tokens has 2^9 times the others' V scale, for the sake of one dimension: the other dimensions'
    values, in its tile and in the others, keep their share. The weights of the digits are P times V scale, so
    max|V| is the outlier's, 2^9 times a usual one, within its tile and nowhere else."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(7200 + D)
    Hkv, G, page, T = 2, 4, 16, 8192
    lens = [100, 1000, 8192, 5000] * 8
    k = torch.randint(-40, 41, (T, Hkv, D), generator=g, device=dev).float()
    v = 64 + 8.0 * torch.randn(T, Hkv, D, generator=g, device=dev)
    vs = torch.full((T // page, 1, Hkv), 2.0 ** -6, device=dev)
    vs[3] *= 2.0 ** 9
    v[48:64] = 0
    v[48:64, :, 5] = 100.0
    kc, vc = [codes_of(t, kind).view(T // page, page, Hkv, D).contiguous() for t in (k, v)]
    ks = torch.full_like(vs, 2.0 ** -6)
    q = torch.randn(len(lens), Hkv * G, D, generator=g, device=dev).to(torch.bfloat16)
    bt = torch.arange(T // page, dtype=torch.int32, device=dev).expand(len(lens), -1).contiguous()
    o, _ = ab.decode_paged_q8(q, kc, vc, ks, vs, bt, torch.tensor(lens, dtype=torch.int32, device=dev))
    vv = values(vc).view(T, Hkv, D) * vs.repeat_interleave(page, 1).view(T, Hkv, 1).double()
    kk = values(kc).view(T, Hkv, D) * 2.0 ** -6
    ref, _, a = reference(q, kk, vv, lens)
    # each dimension's own largest |code| times the largest P * scale of a tile: the outlier's tile has
    # 2^9 * 2^-6 * P <= 8 * P, its P (of 16 tokens) are bounded here by the outlier's own share of dimension 5
    p_out = a[..., 5:6] / (96.0 * 8.0)                         # >= the outlier tokens' largest P (100 is 96 in E4M3)
    code = values(vc).view(T, Hkv, D).abs().amax(0).repeat_interleave(G, 0)
    own = (2.0 ** -9 if kind == "e4m3" else 0.0) + 2.0 ** -14
    bound = 2.0 ** -8 * ref.abs() + own * a + 2.0 ** -15 * (8.0 * p_out + 2.0 ** -6) * code
    err = (o.double() - ref).abs()
    print(kind, D, "error / bound", float((err / bound).max()), "relative", float((err / ref.abs())[..., :5].max()))
    assert (err <= bound).all()
