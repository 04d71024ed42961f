"""The 8-bit cache on the CPU: the oracle's quantiser and attention against independent
statements of the same formulas, and the C ABI's and the binding's refusals (no kernel runs)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import attention_online_softmax_fwd_b200 as ab
from attention_online_softmax_fwd_b200 import binding, build
from attention_online_softmax_fwd_b200 import inputs as gen
from oracle import attn_oracle as orc

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
FAKE = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced on the host


def at(offset):
    return ctypes.c_void_p((1 << 20) + offset)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


# ------------------------------------------------------------------ oracle

def test_e4m3_rounding_matches_torch():
    g = torch.Generator().manual_seed(6000)
    x = torch.randn(50000, generator=g) * torch.exp(3 * torch.randn(50000, generator=g))
    x = torch.cat([x, torch.tensor([0.0, -0.0, 448.0, -448.0, 464.0, 1e9, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(orc.q8_round(x.double().numpy(), "uint8"), want)


@pytest.mark.parametrize("kind", ["uint8", "int8"])
def test_every_code_rounds_to_itself(kind):
    codes = np.array([c for c in range(256) if kind == "int8" or c & 127 != 127], dtype=np.uint8)
    codes = codes.view(np.int8) if kind == "int8" else codes
    codes = codes[codes != -128] if kind == "int8" else codes
    assert np.array_equal(orc.q8_round(orc.q8_values(codes), kind), codes)


@pytest.mark.parametrize("kind,q", [("uint8", 448.0), ("int8", 127.0)])
def test_block_scale_is_the_smallest_power_of_two(kind, q):
    for amax in [0.0, 1e-40, q, np.nextafter(q, 1e9), q / 2, 1.0, 3.3e38, 2.0 ** -95, q * 2.0 ** -100]:
        s = orc.q8_block_scale(amax, kind)
        assert math.frexp(s)[0] == 0.5 and s >= 2.0 ** -100 and q * s < 3.4e38     # every code reads as finite
        assert amax <= q * s or s == orc.Q8_MAX_SCALE[kind]
        assert s == 2.0 ** -100 or amax > q * s / 2
    assert math.isnan(orc.q8_block_scale(float("nan"), kind)) and math.isnan(orc.q8_block_scale(float("inf"), kind))


@pytest.mark.parametrize("kind", ["uint8", "int8"])
def test_append_token_by_token_reads_back_within_half_a_step(kind):
    """One token at a time, sizes growing: each cached value is off by the roundings it went through. A
    value is rounded once when written and once more for each growth of its block's scale (16 tokens grow
    by 4x per token here, so at most 2 binades each), each time by at most half a step of that time's scale."""
    rng = np.random.default_rng(6001)
    Hkv, D, page, block, T = 2, 64, 32, 16, 40
    codes = np.zeros((3, page, Hkv, D), np.uint8 if kind == "uint8" else np.int8)
    scales = np.full((3, page // block, Hkv), 7.0)
    bt = np.array([[2, 0]], np.int32)
    kc, vc, ks, vs = codes, codes.copy(), scales, scales.copy()
    x = torch.tensor(rng.standard_normal((1, T, Hkv, D)) * 1.05 ** np.arange(T)[None, :, None, None]).to(torch.bfloat16)
    for t in range(T):
        kc, vc, ks, vs = orc.kv_append_q8(kc, vc, ks, vs, bt, np.array([t]), x[:, t:t + 1], -x[:, t:t + 1])
    whole = orc.kv_append_q8(codes, codes, scales, scales, bt, np.array([0]), x, -x)
    got = np.concatenate([orc.q8_dequant(kc, ks)[2], orc.q8_dequant(kc, ks)[0]])[:T]
    want = x[0].double().numpy()
    once = np.concatenate([orc.q8_dequant(whole[0], whole[2])[2], orc.q8_dequant(whole[0], whole[2])[0]])[:T]
    s = np.repeat(np.concatenate([ks[2], ks[0]]), block, axis=0)[:T, :, None]      # the final, largest scales
    # half a step relative to the value (E4M3, subnormals: half of 2^-9 in scale units) or of one unit (int8);
    # growths: a scale that starts g binades lower has steps at most 2^-1 of the next one, so the sum of all
    # roundings is below twice the last
    half = np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -10) if kind == "uint8" else s * 0.5
    assert (np.abs(once - want) <= half).all()
    assert (np.abs(got - want) <= 2 * half).all()
    assert np.array_equal(ks, whole[2]) and np.array_equal(vs, whole[3])           # the scales end up the same
    assert np.array_equal(np.abs(orc.q8_values(kc)), np.abs(orc.q8_values(vc)))


def test_append_leaves_everything_else_alone():
    rng = np.random.default_rng(6002)
    codes = rng.integers(-127, 128, (4, 16, 3, 64)).astype(np.int8)
    scales = np.exp2(rng.integers(-8, 0, (4, 1, 3)).astype(float))
    bt = np.array([[1, 3]], np.int32)
    new = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    kc, vc, ks, vs = orc.kv_append_q8(codes, codes, scales, scales, bt, np.array([15]), new, new)
    keep = np.ones_like(codes, bool)
    keep[1, 15], keep[3, 0] = False, False
    assert np.array_equal(kc[keep], codes[keep]) and (kc[~keep] == 0).all()
    assert np.array_equal(ks[[0, 1, 2]], scales[[0, 1, 2]]) and (ks[3] == 2.0 ** -100).all()
    with pytest.raises(IndexError):
        orc.kv_append_q8(codes, codes, scales, scales, bt, np.array([31]), new, new)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_decode_and_prefill_are_the_dense_ones_of_the_read_back_cache(kind):
    cache = gen.paged_decode_inputs(3, 4, 2, 64, 32, 0, 0, seed=6003, lens=[5, 70, 33], poison=False)
    kc, ks = gen.quantize_pool_q8(cache.k_pages, 16, kind)
    vc, vs = gen.quantize_pool_q8(cache.v_pages, 16, kind)
    o, lse = orc.decode_paged_q8(cache.q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, 0.125)
    k, v = orc.q8_dequant(kc, ks), orc.q8_dequant(vc, vs)
    for b, L in enumerate([5, 70, 33]):
        ids = cache.block_table[b, :-(-L // 32)].numpy()
        kk, vv = k[ids].reshape(-1, 2, 64)[:L], v[ids].reshape(-1, 2, 64)[:L]
        qq = cache.q[b].double()
        s = torch.nn.functional.scaled_dot_product_attention(
            qq[None, :, None], torch.tensor(kk).permute(1, 0, 2)[None], torch.tensor(vv).permute(1, 0, 2)[None],
            scale=0.125, enable_gqa=True)
        assert np.abs(o[b] - s[0, :, 0].numpy()).max() < 1e-12
    q = cache.q[:, None]
    op, lp = orc.prefill_paged_q8(q, kc, vc, ks, vs, cache.block_table, cache.seq_lens, 0.125)
    assert np.abs(op[:, 0] - o).max() < 1e-12 and np.abs(lp[:, :, 0] - lse).max() < 1e-12


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_seeded_quantiser_agrees_with_the_oracle(kind):
    g = torch.Generator().manual_seed(6004)
    pool = (torch.randn(3, 64, 2, 64, generator=g) * 3).to(torch.bfloat16)
    codes, scales = gen.quantize_pool_q8(pool, 32, kind)
    z = np.zeros((3, 64, 2, 64), codes.numpy().dtype)
    want = orc.kv_append_q8(z, z, np.ones((3, 2, 2)), np.ones((3, 2, 2)), np.array([[0], [1], [2]]),
                            np.zeros(3, int), pool, pool)
    assert np.array_equal(codes.numpy(), want[0]) and np.array_equal(scales.double().numpy(), want[2])


# ------------------------------------------------------------------ refusals of the C ABI

def _pool(**kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE, fmt=0, N=4, Hkv=3, D=128, ps=32, sb=16, mp=8, P=64,
             ws=FAKE, wsb=1 << 32, scale=0.09)
    a.update(kw)
    return a


def _append(lib, **kw):
    a = _pool(kn=FAKE, vn=FAKE, T=5) | kw
    return lib.attn_kv_append_q8(a["kn"], a["vn"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["fmt"],
                                 a["N"], a["T"], a["Hkv"], a["D"], a["ps"], a["sb"], a["mp"], a["P"], None, None)


def _read(lib, **kw):
    a = _pool(ko=FAKE, vo=FAKE, T=100) | kw
    return lib.attn_kv_read_q8(a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["ko"], a["vo"], a["fmt"],
                               a["N"], a["T"], a["Hkv"], a["D"], a["ps"], a["sb"], a["mp"], a["P"], None, None)


def _decode(lib, **kw):
    a = _pool(q=FAKE, o=FAKE, lse=None, Hq=9) | kw
    return lib.attn_decode_paged_q8(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["fmt"], a["N"],
                                    a["Hq"], a["Hkv"], a["D"], a["ps"], a["sb"], a["mp"], a["P"], a["scale"],
                                    a["o"], a["lse"], a["ws"], a["wsb"], None, None)


def _prefill(lib, **kw):
    a = _pool(q=FAKE, o=FAKE, lse=None, Hq=9, Sq=20) | kw
    return lib.attn_prefill_paged_q8(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["sl"], a["o"], a["lse"],
                                     a["fmt"], a["N"], a["Sq"], a["Hq"], a["Hkv"], a["D"], a["ps"], a["sb"], a["mp"],
                                     a["P"], a["scale"], a["ws"], a["wsb"], None, None)


SHARED_BAD = [dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(sl=None),
              dict(kc=at(8)), dict(vc=at(4)), dict(ks=at(2)), dict(vs=at(1)), dict(bt=at(2)), dict(sl=at(1)),
              dict(fmt=2), dict(fmt=-1), dict(N=0), dict(Hkv=0), dict(ps=24), dict(ps=8), dict(ps=512),
              dict(sb=8), dict(sb=24), dict(sb=64), dict(mp=0), dict(P=0), dict(mp=1 << 26)]


@pytest.mark.parametrize("bad", SHARED_BAD)
@pytest.mark.parametrize("call", [_append, _read, _decode, _prefill])
def test_pool_arguments_are_checked(lib, call, bad):
    assert call(lib, **bad) == INVALID


@pytest.mark.parametrize("call", [_append, _read, _decode, _prefill])
@pytest.mark.parametrize("bad", [dict(D=96), dict(D=256)])
def test_head_dims_are_checked(lib, call, bad):
    assert call(lib, **bad) == UNSUPPORTED


def test_wide_token_rows_are_refused(lib):
    assert _append(lib, Hkv=1 << 14) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(kn=None), dict(vn=None), dict(kn=at(8)), dict(T=0)])
def test_append_refusals(lib, bad):
    assert _append(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(ko=None), dict(vo=at(2)), dict(T=0), dict(T=257)])
def test_read_refusals(lib, bad):
    assert _read(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(q=None), dict(o=None), dict(ws=None), dict(q=at(8)), dict(ws=at(4)),
                                 dict(lse=at(2)), dict(Hq=0), dict(Hq=8), dict(scale=0.0),
                                 dict(scale=float("nan")), dict(wsb=256)])
def test_decode_refusals(lib, bad):
    assert _decode(lib, **bad) == INVALID


def test_decode_refuses_more_than_sixteen_heads_a_group(lib):
    assert _decode(lib, Hq=51, Hkv=3) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(q=None), dict(o=None), dict(ws=None), dict(q=at(8)), dict(lse=at(2)),
                                 dict(Hq=0), dict(Hq=8), dict(Sq=0), dict(Sq=257), dict(scale=-1.0),
                                 dict(scale=float("inf")), dict(wsb=1000)])
def test_prefill_refusals(lib, bad):
    assert _prefill(lib, **bad) == INVALID


def test_valid_arguments_without_a_device_report_cuda_error(lib):
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for call in (_append, _read, _decode, _prefill):
        for fmt in (0, 1):
            assert call(lib, fmt=fmt) == CUDA


def test_prefill_workspace_bytes(lib):
    # bf16 K and V of every page of the table, V behind K at a multiple of 256 bytes, and behind them an LSE and
    # a row of fp32 O for each of 160 CTAs' 256 query rows
    up = lambda x: -(-x // 256) * 256
    for n, hkv, d, mp, ps in [(1, 1, 64, 1, 16), (4, 8, 128, 37, 16), (3, 5, 64, 3, 256)]:
        pool = n * mp * ps * hkv * d * 2
        want = up(up(pool) + pool) + 160 * 256 * (d + 1) * 4
        assert lib.attn_prefill_paged_q8_workspace_bytes(n, hkv, d, mp, ps) == want
        assert binding.prefill_paged_q8_workspace_bytes(n, hkv, d, mp, ps) == want
    for bad in [(0, 8, 128, 4, 16), (1, 0, 128, 4, 16), (1, 8, 96, 4, 16), (1, 8, 128, 0, 16), (1, 8, 128, 4, 24),
                (2 ** 20, 8, 128, 2 ** 20, 16)]:
        assert lib.attn_prefill_paged_q8_workspace_bytes(*bad) == 0


def test_decode_workspace_bytes(lib):
    # {cut sequence} of 16 bytes for each of 320 CTAs; a log2-sum-exp and fp32 O for each of their two parts and
    # its query rows (those of two heads where D = 64 and a group has at most 8), parts padded to 256 bytes
    up = lambda x: -(-x // 256) * 256
    for hq, hkv, d, rows in [(32, 8, 128, 4), (1, 1, 128, 1), (48, 3, 128, 16), (12, 12, 64, 2), (64, 8, 64, 16),
                             (9, 1, 64, 9)]:
        want = up(up(320 * 16) + 640 * rows * 4) + 640 * rows * d * 4
        assert lib.attn_decode_paged_q8_workspace_bytes(hq, hkv, d) == want
        assert binding.decode_paged_q8_workspace_bytes(hq, hkv, d) == want
    for bad in [(0, 1, 128), (4, 0, 128), (9, 2, 128), (4, 2, 96), (34, 2, 128)]:
        assert lib.attn_decode_paged_q8_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ refusals of the binding (CPU tensors)

def test_binding_refuses_host_tensors_and_wrong_types():
    cache = gen.paged_decode_inputs(2, 4, 2, 64, 32, 0, 0, seed=6005, lens=[5, 40], poison=False)
    kc, ks = gen.quantize_pool_q8(cache.k_pages, 16)
    bt, sl = cache.block_table, cache.seq_lens
    with pytest.raises(ab.AttnError, match="CUDA"):
        ab.decode_paged_q8(cache.q, kc, kc, ks, ks, bt, sl)
    with pytest.raises(ab.AttnError, match="uint8"):
        ab.kv_read_q8(kc.float(), kc, ks, ks, bt, sl)
    with pytest.raises(ab.AttnError):
        ab.kv_append_q8(cache.q[:, None], cache.q[:, None], kc, kc, ks, ks, bt, sl)
