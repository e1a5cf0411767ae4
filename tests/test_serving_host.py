"""CPU checks of the attention layers' operators and the block norms: the
rotary frequencies, what the C ABI and the Python binding refuse before
anything is enqueued, and the 64-bit references the GPU tests compare with."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_token_amd as gdn
import serving_ref as ref

INV, UNS, CAP = gdn.GDN_ERR_INVALID, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_CAPACITY
A = 0x100000000
P = [A + i * 0x40000000 for i in range(16)]      # fake, aligned device addresses far apart


# ------------------------------------------------------------- frequencies

def test_plain_frequencies():
    f, m = gdn.gdn_rope_frequencies(64, 1e6)
    assert m == 1.0 and f.shape == (32,)
    np.testing.assert_allclose(f, 1e6 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)


def test_linear_and_ntk_frequencies():
    plain, _ = gdn.gdn_rope_frequencies(128, 1e4)
    lin, m = gdn.gdn_rope_frequencies(128, 1e4, "linear", 8.0)
    assert m == 1.0
    np.testing.assert_allclose(lin, plain / 8, rtol=1e-15)
    ntk, _ = gdn.gdn_rope_frequencies(128, 1e4, "ntk", 4.0)
    assert ntk[0] == 1.0                                   # the fastest pair is left alone,
    np.testing.assert_allclose(ntk[-1], plain[-1] / 4, rtol=1e-12)   # the slowest interpolated in full


def test_yarn_frequencies():
    plain, _ = gdn.gdn_rope_frequencies(128, 1e6)
    f, m = gdn.gdn_rope_frequencies(128, 1e6, "yarn", 4.0, original_context=32768)
    np.testing.assert_allclose(m, 0.1 * math.log(4.0) + 1.0, rtol=1e-15)
    r = ref.turns(plain, 32768)
    fast, slow = r >= 32, r <= 1
    assert fast.any() and slow.any() and not (fast | slow).all()
    np.testing.assert_allclose(f[fast], plain[fast], rtol=1e-15)
    np.testing.assert_allclose(f[slow], plain[slow] / 4, rtol=1e-15)
    ramp = ~(fast | slow)
    assert (f[ramp] < plain[ramp]).all() and (f[ramp] > plain[ramp] / 4).all()


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=63), dict(rotary_dim=0), dict(base=1.0), dict(base=math.nan), dict(scaling="linear", factor=0.5),
    dict(scaling="ntk", factor=2.0, rotary_dim=2), dict(scaling="yarn", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_context=4096, beta_fast=1.0, beta_slow=1.0),
    dict(scaling="yarn", factor=math.inf, original_context=4096),
])
def test_frequencies_refused(kw):
    a = dict(rotary_dim=64, base=1e4)
    a.update(kw)
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_rope_frequencies(**a)
    assert e.value.code == INV


def test_unknown_scaling():
    with pytest.raises(ValueError, match="scaling"):
        gdn.gdn_rope_frequencies(64, 1e4, "cubic")


# ---------------------------------------------------------- the C boundary

def tables(**kw):
    a = dict(ctx=P[0], new=P[1], S=32, free=P[2], nfree=P[3], F=100, bt=P[4], bts=64, cols=64, page=16, qsl=P[5], seq=P[6],
             pos=P[7], slot=P[8], T=40, ch=P[9], nch=37, cnt=P[10])
    a.update(kw)
    return gdn.lib.gdn_build_step_tables(a["ctx"], a["new"], a["S"], a["free"], a["nfree"], a["F"], a["bt"], a["bts"],
                                         a["cols"], a["page"], a["qsl"], a["seq"], a["pos"], a["slot"], a["T"], a["ch"],
                                         a["nch"], a["cnt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(ctx=None), INV), (dict(new=None), INV), (dict(bt=None), INV), (dict(seq=None), INV), (dict(qsl=None), INV),
    (dict(pos=None), INV), (dict(slot=None), INV), (dict(cnt=None), INV), (dict(nfree=None), INV), (dict(free=None), INV),
    (dict(S=-1), INV), (dict(T=-1), INV), (dict(F=-1), INV), (dict(nch=-1), INV), (dict(ch=None), INV), (dict(nch=0), INV),
    (dict(page=0), INV), (dict(page=24), INV), (dict(page=2048), INV), (dict(cols=0), INV), (dict(bts=63), INV),
    (dict(S=4097), UNS), (dict(slot=P[8] + 4), UNS), (dict(ch=P[9] + 4), UNS), (dict(bt=P[4] + 2), UNS),
    (dict(qsl=P[0]), INV), (dict(pos=P[8]), INV), (dict(cnt=P[5] + 4 * 32), INV), (dict(bt=P[2] + 4 * 99), INV),
])
def test_tables_refusals(kw, code):
    assert tables(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


def rope(**kw):
    a = dict(q=P[0], qs=4096, k=P[1], ks=1024, v=P[2], vs=1024, pos=P[3], slot=P[4], f=P[5], rot=64, il=0, m=1.0, qo=P[6],
             qos=4096, kc=P[7], vc=P[8], ksc=P[9], vsc=P[10], n=64, page=16, T=8, HQ=16, HK=4, D=256)
    a.update(kw)
    return gdn.lib.gdn_rope_append_kv8(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["slot"], a["f"], a["rot"],
                                       a["il"], a["m"], a["qo"], a["qos"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["n"],
                                       a["page"], a["T"], a["HQ"], a["HK"], a["D"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(pos=None), INV), (dict(slot=None), INV), (dict(f=None), INV),
    (dict(q=None), INV), (dict(qo=None), INV), (dict(kc=None), INV), (dict(vsc=None), INV), (dict(T=-1), INV),
    (dict(n=0), INV), (dict(HQ=0), INV), (dict(HK=0), INV), (dict(qs=4088), INV), (dict(ks=1016), INV), (dict(qos=8), INV),
    (dict(page=8), UNS), (dict(page=48), UNS), (dict(D=96), UNS), (dict(rot=8), UNS), (dict(rot=272), UNS), (dict(rot=-16), UNS),
    (dict(ks=1028), UNS), (dict(q=P[0] + 2), UNS), (dict(kc=P[7] + 8), UNS), (dict(slot=P[4] + 4), UNS), (dict(f=P[5] + 4), UNS),
    (dict(qo=P[0] + 16), INV), (dict(qo=P[1]), INV), (dict(qo=P[0], qos=4104), INV), (dict(kc=P[8]), INV), (dict(ksc=P[7]), INV),
    (dict(vc=P[2]), INV), (dict(qo=P[9]), INV),
    # columns of one projection row: q_out over k's columns
    (dict(q=P[0], qs=6144, k=P[0] + 2 * 4096, ks=6144, v=P[0] + 2 * 5120, vs=6144, qo=P[0] + 2 * 1024, qos=6144), INV),
])
def test_rope_append_refusals(kw, code):
    assert rope(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


@pytest.mark.parametrize("kw", [dict(ks=1 << 24), dict(vs=1 << 24), dict(ks=(1 << 24) + 8, vs=(1 << 24) + 8)])
def test_rope_append_refuses_far_strides(kw):
    # a page's rows are addressed with 32-bit offsets
    assert rope(**kw) == UNS and b"2^24" in gdn.lib.gdn_last_error()


def attn(**kw):
    a = dict(q=P[0], qs=4096, kc=P[1], vc=P[2], ksc=P[3], vsc=P[4], n=64, page=16, bt=P[5], bts=32, cols=32, seq=P[6], qsl=P[7],
             longest=500, o=P[8], os=4096, S=2, T=8, HQ=16, HK=4, D=256, scale=1.0, causal=1, window=0, ws=P[9], wsn=1 << 28)
    a.update(kw)
    return gdn.lib.gdn_paged_attention_kv8(a["q"], a["qs"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["n"], a["page"], a["bt"],
                                           a["bts"], a["cols"], a["seq"], a["qsl"], a["longest"], a["o"], a["os"], a["S"],
                                           a["T"], a["HQ"], a["HK"], a["D"], a["scale"], a["causal"], a["window"], a["ws"],
                                           a["wsn"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(o=None), INV), (dict(bt=None), INV), (dict(seq=None), INV), (dict(qsl=None), INV),
    (dict(kc=None), INV), (dict(ksc=None), INV), (dict(S=-1), INV), (dict(T=-1), INV), (dict(n=0), INV), (dict(HQ=6), INV),
    (dict(HQ=0), INV), (dict(HK=0), INV), (dict(cols=0), INV), (dict(bts=31), INV), (dict(longest=0), INV), (dict(window=-1), INV),
    (dict(qs=4088), INV), (dict(os=64), INV), (dict(page=128), UNS), (dict(D=32), UNS), (dict(os=4100), UNS), (dict(o=P[8] + 4), UNS),
    (dict(cols=1 << 28, bts=1 << 28), UNS), (dict(o=P[0]), INV), (dict(o=P[1]), INV), (dict(o=P[6]), INV), (dict(seq=P[6] + 1), UNS),
])
def test_attention_refusals(kw, code):
    assert attn(**kw) == code, gdn.lib.gdn_last_error()
    assert gdn.lib.gdn_last_error()


def head(**kw):
    a = dict(x=P[0], xs=4096, g=P[1], gs=4096, w=P[2], y=P[3], ys=4096, T=8, H=32, D=128)
    a.update(kw)
    return gdn.lib.gdn_gated_rms_norm(a["x"], a["xs"], a["g"], a["gs"], a["w"], a["y"], a["ys"], a["T"], a["H"], a["D"], 1e-6, 0.0,
                                      None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(xs=8), INV),
    (dict(gs=8), INV), (dict(ys=8), INV), (dict(D=100), UNS), (dict(D=520, H=1), UNS), (dict(D=0), UNS), (dict(xs=4100), UNS),
    (dict(y=P[3] + 8), UNS), (dict(y=P[0] + 16), INV), (dict(y=P[0], ys=4104), INV), (dict(y=P[1]), INV), (dict(w=P[3]), INV),
])
def test_head_norm_refusals(kw, code):
    assert head(**kw) == code, gdn.lib.gdn_last_error()


def resid(**kw):
    a = dict(x=P[0], xs=2560, r=P[1], rs=2560, pw=P[2], g=P[3], gs=2560, w=P[4], n=P[5], ns=2560, y=P[6], ys=2560, R=4, D=2560)
    a.update(kw)
    return gdn.lib.gdn_residual_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["pw"], a["g"], a["gs"], a["w"], a["n"], a["ns"],
                                         a["y"], a["ys"], a["R"], a["D"], 1.0, 1e-6, 0.0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(r=None), INV), (dict(w=None), INV), (dict(n=None), INV), (dict(y=None), INV), (dict(R=-1), INV),
    (dict(xs=2552), INV), (dict(rs=2552), INV), (dict(gs=8), INV), (dict(ns=8), INV), (dict(ys=8), INV), (dict(D=2556), UNS),
    (dict(D=16392, xs=16392, rs=16392, gs=16392, ns=16392, ys=16392), UNS), (dict(D=0), UNS), (dict(xs=2564), UNS),
    (dict(pw=P[2] + 2), UNS), (dict(y=P[5]), INV), (dict(y=P[1]), INV), (dict(y=P[3]), INV), (dict(n=P[3]), INV),
    (dict(n=P[1] + 16), INV), (dict(n=P[1], ns=2568), INV), (dict(y=P[4]), INV), (dict(n=P[2]), INV),
])
def test_residual_norm_refusals(kw, code):
    assert resid(**kw) == code, gdn.lib.gdn_last_error()


def test_calls_without_tokens_enqueue_nothing():
    assert rope(T=0, k=None, q=None) == 0 and attn(T=0, q=None) == 0 and attn(S=0, bt=None) == 0
    assert head(T=0, x=None) == 0 and resid(R=0, x=None) == 0


def test_workspace_size_of_nothing_is_zero():
    size = gdn.gdn_paged_attention_kv8_workspace_size
    assert size(0, 1, 8, 1, 64, 100) == 0 and size(1, 0, 8, 1, 64, 100) == 0 and size(1, 1, 8, 3, 64, 100) == 0
    assert size(1, 1, 8, 1, 64, 0) == 0 and size(-1, 1, 8, 1, 64, 9) == 0


# --------------------------------------------------------- the Python binding

class _Recorder:
    """Stands in for the library: records every call instead of making it."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_workspace_size") or name == "gdn_last_error":
            return getattr(self.real, name)
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(gdn.lib)
    monkeypatch.setattr(gdn, "lib", r)
    yield r
    assert r.calls == [], "the library was called: %s" % r.calls


BF, F32, I32, I64, F8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=torch.uint8).view(F8) if dtype == F8 else torch.zeros(*shape, dtype=dtype)


def cache(n=6, hk=2, page=16, d=64):
    return dict(k_cache=z(n, hk, page, d, dtype=F8), v_cache=z(n, hk, d, page, dtype=F8), k_scale=z(n, hk, dtype=F32),
                v_scale=z(n, hk, dtype=F32))


def tables_args():
    return dict(context_lens=z(3, dtype=I32), query_lens=z(3, dtype=I32), free_pages=z(9, dtype=I32), num_free=z(1, dtype=I32),
                block_table=z(3, 5, dtype=I32), page_size=16, query_start_loc=z(4, dtype=I32), seq_lens=z(3, dtype=I32),
                positions=z(7, dtype=I32), slot_mapping=z(7, dtype=I64), counts=z(4, dtype=I32), chunks=z(4, 2, dtype=I32))


@pytest.mark.parametrize("change,msg", [
    (dict(), "GPU tensor"), (dict(query_lens=z(2, dtype=I32)), "query_lens"), (dict(block_table=z(2, 5, dtype=I32)), "block_table"),
    (dict(block_table=z(3, 5, dtype=I64)), "block_table"), (dict(query_start_loc=z(3, dtype=I32)), "query_start_loc"),
    (dict(slot_mapping=z(7, dtype=I32)), "slot_mapping"), (dict(slot_mapping=z(6, dtype=I64)), "slot_mapping"),
    (dict(counts=z(3, dtype=I32)), "counts"), (dict(chunks=z(4, 3, dtype=I32)), "chunks"), (dict(num_free=z(2, dtype=I32)), "num_free"),
    (dict(context_lens=z(6, dtype=I32)[::2]), "context_lens"),
])
def test_tables_binding_rejects(rec, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        gdn.gdn_build_step_tables(**{**tables_args(), **change})


def append_args():
    return dict(q=z(7, 4, 64), k=z(7, 2, 64), v=z(7, 2, 64), positions=z(7, dtype=I32), slot_mapping=z(7, dtype=I64),
                frequencies=z(16, dtype=torch.float64), q_out=z(7, 4, 64), **cache())


@pytest.mark.parametrize("change,msg", [
    (dict(), "GPU tensor"), (dict(k=z(7, 3, 64)), "k must"), (dict(v=z(6, 2, 64)), "v must"), (dict(q=None), "q and q_out"),
    (dict(q_out=z(7, 4, 32)), "q_out"), (dict(q=z(7, 4, 64, dtype=F32)), "q must"), (dict(positions=z(6, dtype=I32)), "positions"),
    (dict(slot_mapping=z(7, dtype=I32)), "slot_mapping"), (dict(frequencies=z(16, dtype=F32)), "frequencies"),
    (dict(k_cache=z(6, 2, 16, 64, dtype=torch.uint8)), "k_cache"), (dict(v_cache=z(6, 2, 16, 64, dtype=F8)), "v_cache"),
    (dict(k_scale=z(6, 1, dtype=F32)), "k_scale"), (dict(v_scale=z(6, 2, dtype=BF)), "v_scale"),
])
def test_append_binding_rejects(rec, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        gdn.gdn_rope_append_kv8(**{**append_args(), **change})


def attention_args():
    return dict(q=z(7, 4, 64), block_table=z(3, 5, dtype=I32), seq_lens=z(3, dtype=I32), query_start_loc=z(4, dtype=I32),
                o=z(7, 4, 64), max_seq_len=80, scale=0.125, **cache())


@pytest.mark.parametrize("change,msg", [
    (dict(), "GPU tensor"), (dict(o=z(7, 4, 32)), "o must"), (dict(block_table=z(2, 5, dtype=I32)), "block_table"),
    (dict(query_start_loc=z(3, dtype=I32)), "query_start_loc"), (dict(seq_lens=z(3, dtype=I64)), "seq_lens"),
    (dict(q=z(7, 4, 128)), "q must"), (dict(v_cache=z(6, 2, 16, 64, dtype=F8)), "v_cache"),
])
def test_attention_binding_rejects(rec, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        gdn.gdn_paged_attention_kv8(**{**attention_args(), **change})


@pytest.mark.parametrize("change,msg", [
    (dict(), "GPU tensor"), (dict(y=z(5, 2, 32)), "y must"), (dict(gate=z(5, 2, 64, dtype=F32)), "gate"), (dict(weight=z(32)), "weight"),
    (dict(x=z(5, 128)), "x must"),
])
def test_head_norm_binding_rejects(rec, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        gdn.gdn_gated_rms_norm(**{**dict(x=z(5, 2, 64), weight=z(64), y=z(5, 2, 64)), **change})


@pytest.mark.parametrize("change,msg", [
    (dict(), "GPU tensor"), (dict(residual=z(4, 64)), "residual"), (dict(post_weight=z(32)), "post_weight"), (dict(y=z(5, 64, dtype=F32)), "y must"),
    (dict(gate=z(5, 32)), "gate"),
])
def test_residual_norm_binding_rejects(rec, change, msg):
    with pytest.raises((ValueError, TypeError), match=msg):
        gdn.gdn_residual_rms_norm(**{**dict(x=z(5, 64), residual=z(5, 64), weight=z(64), new_residual=z(5, 64), y=z(5, 64)), **change})


# ------------------------------------------------------------ the references

def test_reference_e4m3_matches_torch():
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(1)) * s for s in (1e-3, 0.02, 1.0, 60.0)]).clamp(-448, 448)
    assert np.array_equal(ref.e4m3(x.double().numpy()), x.to(F8).double().numpy())


def test_reference_block_scale():
    for m in (0.0, 1e-30, 447.9, 448.0, 448.1, 1.0, 1.75, 1.7500001, 3e38):
        s = ref.block_scale(m)
        assert m <= 448 * s and (s == 2.0 ** -100 or m > 224 * s)


def test_reference_attention_without_keys_is_zero_and_uniform_is_mean():
    k = np.zeros((2, 1, 16, 4))
    v = np.random.default_rng(0).standard_normal((2, 1, 4, 16))
    one = np.ones((2, 1))
    o, _ = ref.attention(np.ones((3, 1, 4)), k, v, one, one, np.array([[1, 0], [-1, -1]]), [20, 5], [0, 2, 3], 1.0, causal=False)
    full = np.concatenate([v[1, 0], v[0, 0][:, :4]], 1)
    np.testing.assert_allclose(o[0, 0], full.mean(1))
    assert (o[2] == 0).all()
