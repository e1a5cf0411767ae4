"""CPU checks of the 4-bit paged cache: its 64-bit reference, and what the C ABI
and the Python binding refuse before anything is enqueued."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import kv4_ref as kv4

INV, UNS, CAP = gdn.GDN_ERR_INVALID, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_CAPACITY
A = 0x100000000
P = [A + i * 0x40000000 for i in range(16)]      # fake, aligned device addresses far apart


# ------------------------------------------------------------ the reference

def test_codes_are_the_nearest_values():
    x = np.linspace(-8, 8, 100001)
    got = kv4.VALUES[kv4.e2m1(x)]
    best = np.abs(x[:, None] - kv4.VALUES[None]).min(1)
    assert np.array_equal(np.abs(got - x), best)


def test_ties_go_to_the_even_code():
    for lo in range(7):
        middle = (kv4.MAGNITUDES[lo] + kv4.MAGNITUDES[lo + 1]) / 2
        assert kv4.e2m1(middle) % 2 == 0 and kv4.e2m1(-middle) % 2 == 0
    assert kv4.e2m1(100.0) == 7 and kv4.e2m1(-0.0) == 8


def test_key_scales_meet_the_largest_magnitude():
    for m in np.concatenate([np.exp2(np.linspace(-99, 127, 5000)), [1.75, 1.7499, 1.0, 0.875, 2.0 ** 100 * 1.75]]):
        s = 2.0 ** int(kv4.key_exponent(m))
        assert 3.5 * s <= m < 7 * s or s == 2.0 ** -100
    assert kv4.key_exponent(0.0) == -100 and kv4.key_exponent(2.0 ** -140) == -100


def test_no_key_is_off_by_more_than_half_a_step_of_its_binade():
    r = np.random.default_rng(0)
    x = r.standard_normal((3000, 32)) * np.exp(r.standard_normal((3000, 1)))
    codes, scale = kv4.quantise_k(x)
    s = np.exp2(scale.astype(int) - 127.0)
    step = np.maximum(np.exp2(np.floor(np.log2(np.abs(x)))) / 2, s / 2)
    assert (np.abs(kv4.key_values(codes, scale) - x) <= step / 2).all()


def test_value_scales():
    for m in np.exp2(np.random.default_rng(1).uniform(-90, 120, 2000)):
        s = float(kv4.value_scale(m))
        assert abs(s - m / 6) <= m / 6 * 2.0 ** -8 and s == float(torch.tensor(s).to(torch.bfloat16))
        assert kv4.e2m1(m / s) == 7
    assert kv4.value_scale(0.0) == 2.0 ** -100


def test_packing_is_undone():
    r = np.random.default_rng(2)
    c = r.integers(0, 16, (3, 2, 32, 64), dtype=np.uint8)
    assert np.array_equal(kv4.unpack_k(kv4.pack_k(c)), c) and np.array_equal(kv4.unpack_v(kv4.pack_v(c)), c)
    v = kv4.pack_v(c)
    assert v.shape == (3, 2, 2, 64, 8) and v[1, 0, 1, 5, 3] == c[1, 0, 22, 5] | c[1, 0, 23, 5] << 4


def test_three_parts_hold_q():
    """Exact down to 2^-7 of the largest of 32, within 2^-15 of it below."""
    sig = 1 + np.arange(128) / 128
    for top in sig:
        for level in range(16):
            x = np.zeros((128, 32))
            x[:, 3], x[:, 7] = top, np.minimum(sig * 2.0 ** -level, top)
            err = np.abs(kv4.split(x) - x).max()
            assert err <= (0.0 if level <= 7 else 2.0 ** -15 * top)


# ---------------------------------------------------------- the C boundary

def rope(**kw):
    a = dict(q=P[0], qs=4096, k=P[1], ks=1024, v=P[2], vs=1024, pos=P[3], slot=P[4], f=P[5], rot=64, il=0, m=1.0, qo=P[6],
             qos=4096, kc=P[7], vc=P[8], ksc=P[9], vsc=P[10], n=64, page=16, T=8, HQ=16, HK=4, D=256)
    a.update(kw)
    return gdn.lib.gdn_rope_append_kv4(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["slot"], a["f"], a["rot"],
                                       a["il"], a["m"], a["qo"], a["qos"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["n"],
                                       a["page"], a["T"], a["HQ"], a["HK"], a["D"], None)


HEADS = 64 * 4                                    # pages x kv heads of the calls here


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(pos=None), INV), (dict(slot=None), INV), (dict(f=None), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(ksc=None), INV), (dict(vsc=None), INV),
    (dict(T=-1), INV), (dict(n=0), INV), (dict(HQ=0), INV), (dict(HK=0), INV), (dict(qs=4088), INV), (dict(ks=1016), INV),
    (dict(qos=8), INV), (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=128), UNS), (dict(D=96), UNS), (dict(rot=8), UNS),
    (dict(rot=272), UNS), (dict(rot=-16), UNS), (dict(ks=1028), UNS), (dict(vs=1 << 24), UNS), (dict(q=P[0] + 2), UNS),
    (dict(kc=P[7] + 8), UNS), (dict(vc=P[8] + 8), UNS), (dict(ksc=P[9] + 4), UNS), (dict(vsc=P[10] + 8), UNS),
    (dict(slot=P[4] + 4), UNS), (dict(f=P[5] + 4), UNS), (dict(pos=P[3] + 2), UNS),
    (dict(qo=P[0] + 16), INV), (dict(qo=P[1]), INV), (dict(qo=P[0], qos=4104), INV), (dict(kc=P[8]), INV), (dict(ksc=P[7]), INV),
    (dict(vc=P[2]), INV), (dict(qo=P[9]), INV), (dict(vsc=P[7] + HEADS * 16 * 128 - 16), INV), (dict(kc=P[9] + HEADS * 16 * 8 - 16), INV),
    (dict(ksc=P[10] + HEADS * 16 * 2 - 16), INV),
])
def test_append_refusals(kw, code):
    assert rope(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


def read(**kw):
    a = dict(kc=P[0], vc=P[1], ksc=P[2], vsc=P[3], n=64, page=16, bt=P[4], bts=20, cols=20, st=P[5], loc=P[6], k=P[7], ks=1024, v=P[8],
             vs=1024, S=3, R=50, HK=4, D=256)
    a.update(kw)
    return gdn.lib.gdn_paged_read_kv4(a["kc"], a["vc"], a["ksc"], a["vsc"], a["n"], a["page"], a["bt"], a["bts"], a["cols"], a["st"],
                                      a["loc"], a["k"], a["ks"], a["v"], a["vs"], a["S"], a["R"], a["HK"], a["D"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INV), (dict(R=-1), INV), (dict(bt=None), INV), (dict(loc=None), INV), (dict(k=None, v=None), INV), (dict(kc=None), INV),
    (dict(vsc=None), INV), (dict(n=0), INV), (dict(HK=0), INV), (dict(cols=0), INV), (dict(bts=19), INV), (dict(ks=1016), INV),
    (dict(vs=1016), INV), (dict(k=None, vs=1016), INV), (dict(page=24), UNS), (dict(D=80), UNS), (dict(ks=1028), UNS), (dict(vs=1028), UNS),
    (dict(k=P[7] + 8), UNS), (dict(v=P[8] + 2), UNS), (dict(bt=P[4] + 2), UNS), (dict(st=P[5] + 1), UNS), (dict(loc=P[6] + 2), UNS),
    (dict(kc=P[0] + 8), UNS), (dict(vsc=P[3] + 2), UNS), (dict(k=P[8]), INV), (dict(v=P[7] + 1024), INV), (dict(k=P[0]), INV),
    (dict(v=P[1] + HEADS * 16 * 128 - 16), INV), (dict(k=P[2]), INV), (dict(v=P[3]), INV), (dict(st=P[7]), INV), (dict(loc=P[8]), INV),
    (dict(bt=P[8] + 50 * 2048 - 4), INV), (dict(k=P[7], ks=1536, v=P[7] + 1024, vs=1536), INV),
])
def test_read_refusals(kw, code):
    assert read(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


def attn(**kw):
    a = dict(q=P[0], qs=4096, kc=P[1], vc=P[2], ks=P[3], vs=P[4], n=64, page=16, bt=P[5], bts=70, cols=70, seq=P[6], qsl=P[7], longest=1100,
             o=P[8], os=4096, S=32, T=32, HQ=16, HK=4, D=256, scale=0.0625, causal=1, window=0, ws=P[9], wsb=1 << 30)
    a.update(kw)
    return gdn.lib.gdn_paged_attention_kv4(a["q"], a["qs"], a["kc"], a["vc"], a["ks"], a["vs"], a["n"], a["page"], a["bt"], a["bts"],
                                           a["cols"], a["seq"], a["qsl"], a["longest"], a["o"], a["os"], a["S"], a["T"], a["HQ"],
                                           a["HK"], a["D"], a["scale"], a["causal"], a["window"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(o=None), INV), (dict(bt=None), INV), (dict(seq=None), INV), (dict(qsl=None), INV), (dict(kc=None), INV),
    (dict(vs=None), INV), (dict(S=-1), INV), (dict(T=-1), INV), (dict(HQ=6), INV), (dict(HQ=0), INV), (dict(HK=0), INV), (dict(n=0), INV),
    (dict(cols=0), INV), (dict(bts=69), INV), (dict(longest=0), INV), (dict(window=-1), INV), (dict(qs=4088), INV), (dict(os=8), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(scale=-math.inf), INV), (dict(page=8), UNS), (dict(D=96), UNS),
    (dict(cols=2 ** 27, bts=2 ** 27), UNS), (dict(qs=4100), UNS), (dict(q=P[0] + 8), UNS), (dict(o=P[8] + 2), UNS), (dict(ks=P[3] + 4), UNS),
    (dict(vs=P[4] + 2), UNS), (dict(bt=P[5] + 2), UNS), (dict(seq=P[6] + 1), UNS), (dict(o=P[0]), INV), (dict(o=P[1]), INV), (dict(o=P[4]), INV),
    (dict(o=P[2] + HEADS * 16 * 128 - 16), INV),
    # few rows over long contexts: with a workspace
    (dict(S=3, T=3, longest=90000, ws=None), INV), (dict(S=3, T=3, longest=90000, ws=P[9] + 16), UNS),
    (dict(S=3, T=3, longest=90000, wsb=100), CAP), (dict(S=3, T=3, longest=90000, ws=P[0]), INV),
    (dict(S=3, T=3, longest=90000, ws=P[3]), INV), (dict(S=3, T=3, longest=90000, ws=P[8]), INV),
])
def test_attention_refusals(kw, code):
    assert attn(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


def test_calls_without_tokens_enqueue_nothing():
    assert rope(T=0, k=None) == 0 and read(R=0, bt=None) == 0 and read(S=0, kc=None) == 0
    assert attn(T=0, q=None) == 0 and attn(S=0, scale=math.nan) == 0


def test_workspace_size_of_nothing_is_zero():
    size = gdn.gdn_paged_attention_kv4_workspace_size
    assert size(0, 1, 4, 2, 64, 100) == 0 and size(1, 1, 5, 2, 64, 100) == 0 and size(1, 0, 4, 2, 64, 100) == 0
    assert size(1, 1, 4, 2, 64, 100000) > 0


# -------------------------------------------------------------- the binding

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


@pytest.fixture
def rec(monkeypatch):
    """The library's calls recorded, nothing enqueued."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_workspace_size"):
                return lambda *a: 0
            return lambda *a: calls.append((name, a)) or 0

    monkeypatch.setattr(gdn, "lib", Lib())
    monkeypatch.setattr(gdn, "_on_current", lambda names, *t: 0)
    monkeypatch.setattr(gdn, "_stream_on", lambda stream, device: None)
    return calls


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def cache(n=6, hk=2, page=16, d=64):
    return dict(k_cache=z(n, hk, page, d // 2, dtype=U8), v_cache=z(n, hk, page // 16, d, 8, dtype=U8),
                k_scale=z(n, hk, d // 32, page, dtype=U8), v_scale=z(n, hk, page))


BAD_CACHES = [
    (dict(k_cache=z(6, 2, 16, 32, dtype=torch.int8)), TypeError), (dict(v_scale=z(6, 2, 16, dtype=torch.float32)), TypeError),
    (dict(k_scale=z(6, 2, 2, 16, dtype=torch.float32)), TypeError), (dict(k_cache=z(6, 2, 16, dtype=U8)), ValueError),
    (dict(v_cache=z(6, 2, 64, 8, dtype=U8)), ValueError), (dict(v_cache=z(6, 2, 2, 64, 8, dtype=U8)), ValueError),
    (dict(k_scale=z(6, 2, 16, 2, dtype=U8)), ValueError), (dict(v_scale=z(6, 2, 64)), ValueError),
    (dict(k_cache=z(6, 2, 32, 32, dtype=U8)[:, :, ::2]), ValueError),
]


def append_args():
    return dict(q=z(5, 4, 64), k=z(5, 2, 64), v=z(5, 2, 64), positions=z(5, dtype=I32), slot_mapping=z(5, dtype=torch.int64),
                frequencies=z(32, dtype=torch.float64), q_out=z(5, 4, 64), **cache())


@pytest.mark.parametrize("change,error", BAD_CACHES + [
    (dict(q_out=None), ValueError), (dict(q=z(4, 4, 64)), ValueError), (dict(k=z(5, 2, 64, dtype=torch.float16)), TypeError),
    (dict(v=z(5, 3, 64)), ValueError), (dict(positions=z(5, dtype=torch.int64)), TypeError), (dict(slot_mapping=z(4, dtype=torch.int64)), ValueError),
    (dict(frequencies=z(32, dtype=torch.float32)), TypeError),
])
def test_append_binding_rejects(rec, change, error):
    gdn.gdn_rope_append_kv4(**append_args())
    assert [n for n, _ in rec] == ["gdn_rope_append_kv4"]
    with pytest.raises(error):
        gdn.gdn_rope_append_kv4(**{**append_args(), **change})


def read_args():
    return dict(block_table=z(3, 4, dtype=I32), key_starts=z(3, dtype=I32), out_start_loc=z(4, dtype=I32), k_out=z(9, 2, 64), v_out=z(9, 2, 64),
                **cache())


@pytest.mark.parametrize("change,error", BAD_CACHES + [
    (dict(k_out=None, v_out=None), ValueError), (dict(v_out=z(8, 2, 64)), ValueError),
    (dict(k_out=z(9, 3, 64)), ValueError), (dict(k_out=z(9, 2, 64, dtype=torch.float32)), TypeError), (dict(block_table=z(2, 4, dtype=I32)), ValueError),
    (dict(block_table=z(3, 4, dtype=torch.int64)), TypeError), (dict(key_starts=z(4, dtype=I32)), ValueError),
    (dict(out_start_loc=z(4, dtype=torch.int64)), TypeError), (dict(out_start_loc=z(0, dtype=I32)), ValueError),
])
def test_read_binding_rejects(rec, change, error):
    gdn.gdn_paged_read_kv4(**read_args())
    gdn.gdn_paged_read_kv4(**{**read_args(), "key_starts": None, "v_out": None})
    assert len(rec) == 2 and rec[1][1][9] is None and rec[1][1][13] is None
    with pytest.raises(error):
        gdn.gdn_paged_read_kv4(**{**read_args(), **change})


def attention_args():
    return dict(q=z(5, 4, 64), block_table=z(3, 4, dtype=I32), seq_lens=z(3, dtype=I32), query_start_loc=z(4, dtype=I32), o=z(5, 4, 64),
                max_seq_len=64, scale=0.125, **cache())


@pytest.mark.parametrize("change,error", BAD_CACHES + [
    (dict(o=z(5, 2, 64)), ValueError), (dict(q=z(5, 4, 128)), ValueError), (dict(seq_lens=z(3, dtype=torch.int64)), TypeError),
    (dict(query_start_loc=z(3, dtype=I32)), ValueError), (dict(block_table=z(2, 4, dtype=I32)), ValueError),
])
def test_attention_binding_rejects(rec, change, error):
    gdn.gdn_paged_attention_kv4(**attention_args())
    assert [n for n, _ in rec] == ["gdn_paged_attention_kv4"]
    with pytest.raises(error):
        gdn.gdn_paged_attention_kv4(**{**attention_args(), **change})
