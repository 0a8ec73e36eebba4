"""The paged-cache operators without a GPU: the host code and the kernels' index arithmetic
under sanitizers, the refusals of the binding, the rotary frequencies, the oracle itself."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle.kv_oracle as KO
import rank_adapter_gemm_build_amd as rx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "rank_adapter_gemm_build_amd", "csrc")


def test_kv_host_code_and_index_arithmetic_under_asan_ubsan(tmp_path):
    gxx = shutil.which("g++")
    if not gxx or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ or the ROCm headers are missing")
    exe = str(tmp_path / "kv_sanitized")
    flags = ["address", "undefined"]
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=" + ",".join(flags),
           "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "api.cpp"), os.path.join(CSRC, "kv.cpp"),
           os.path.join(HERE, "hip_stubs.cpp"), os.path.join(HERE, "kv_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-6000:])
    assert r.stdout.strip().endswith("0 failures")


# ------------------------------------------------------------------------- frequencies
# one term of pow, log and a product each differ by a few units in the last place: 2^-45
# relative is a thousand of them; a blend weight differs by that much absolutely
@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="wavelength", factor=8.0, original_len=8192, low=1, high=4),
    dict(scaling="dim", factor=16.0, original_len=4096, low=1, high=32), dict(scaling="dim", factor=2.0, original_len=16, low=1, high=2),
    dict(scaling="wavelength", factor=1.0, original_len=100, low=0.5, high=100),
])
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6), (20, 2.0)])
def test_frequencies(rot, base, kw):
    got = rx.rotary_frequencies(rot, base, **kw)
    want = KO.frequencies(rot, base, kw.get("scaling", "plain"), kw.get("factor", 1.0), kw.get("original_len", 0),
                          kw.get("low", 0), kw.get("high", 0))
    assert len(got) == rot // 2
    np.testing.assert_allclose(got, want, rtol=2.0 ** -45 * kw.get("factor", 1.0) * 16)


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=300), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, scaling="linear", factor=0.0),
                                dict(rot_dim=64, scaling="dim", factor=2.0, original_len=0.0, low=1, high=32)])
def test_frequencies_refused(kw):
    with pytest.raises(rx.LoraError):
        rx.rotary_frequencies(**kw)


def test_unknown_scaling_refused():
    with pytest.raises(ValueError):
        rx.rotary_frequencies(64, scaling="other")


def test_exported_constants():
    text = open(os.path.join(ROOT, "include", "raxlora.h")).read()
    for name in ("LORA_MAX_SEQS", "LORA_MAX_HEAD_DIM", "LORA_PLAN_META"):
        assert re.search(rf"#define\s+{name}\s+{getattr(rx, name)}\b", text), name


def test_missing_device_is_reported():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for make in (lambda: rx.Rotary(0, 64, rx.rotary_frequencies(64)), lambda: rx.Attention(0, 4, 8, 8, 2, 64)):
        with pytest.raises(rx.LoraError) as e:
            make()
        assert e.value.status in (rx.LORA_ERR_NO_DEVICE, rx.LORA_ERR_HIP)


# ------------------------------------------------------------------------- the binding
BF = torch.bfloat16


def _cpu_cache(**kw):
    return rx.KVCache(torch.zeros(4, 16, 2, 32, dtype=kw.pop("dtype", BF)), torch.zeros(4, 16, 2, 32, dtype=kw.pop("vdtype", BF)), **kw)


@pytest.mark.parametrize("make,err", [
    (lambda: rx.KVCache(torch.zeros(4, 16, 2, 32, dtype=BF), np.zeros((4, 16, 2, 32))), TypeError),
    (lambda: rx.KVCache(torch.zeros(4, 16, 64, dtype=BF), torch.zeros(4, 16, 64, dtype=BF)), ValueError),
    (lambda: _cpu_cache(vdtype=torch.float32), ValueError),
    (lambda: _cpu_cache(dtype=torch.float16, vdtype=torch.float16), TypeError),
    (lambda: rx.KVCache(torch.zeros(4, 12, 2, 32, dtype=BF), torch.zeros(4, 12, 2, 32, dtype=BF)), ValueError),
    (lambda: rx.KVCache(torch.zeros(4, 16, 2, 40, dtype=BF), torch.zeros(4, 16, 2, 40, dtype=BF)), ValueError),
    (lambda: rx.KVCache(torch.zeros(4, 16, 2, 272, dtype=BF), torch.zeros(4, 16, 2, 272, dtype=BF)), ValueError),
    (lambda: rx.KVCache(torch.zeros(4, 16, 32, 2, dtype=BF).transpose(2, 3), torch.zeros(4, 16, 32, 2, dtype=BF).transpose(2, 3)),
     ValueError),
    (lambda: rx.KVCache(torch.zeros(4, 2, 16, 32, dtype=BF).transpose(1, 2), torch.zeros(4, 16, 2, 32, dtype=BF)), ValueError),
    (lambda: rx.KVCache(torch.zeros(4, 16, 2, 32, dtype=torch.uint8), torch.zeros(4, 16, 2, 32, dtype=torch.uint8), k_scale=0.0),
     ValueError),
])
def test_cache_refused(make, err):
    with pytest.raises(err):
        make()


def _object(cls, **kw):
    o = object.__new__(cls)
    o.__dict__.update(handle=0, **kw)
    return o


class _NoCalls:
    def __getattr__(self, name):
        raise AssertionError(f"the library was called: {name}")


I32 = torch.int32


@pytest.mark.parametrize("change,err", [
    (dict(qkv=torch.zeros(3, 256)), TypeError), (dict(qkv=torch.zeros(3, 248, dtype=BF)), ValueError),
    (dict(qkv=torch.zeros(256, 3, dtype=BF).t()), ValueError), (dict(q_out=torch.zeros(2, 128, dtype=BF)), ValueError),
    (dict(q_out=torch.zeros(3, 128)), TypeError), (dict(positions=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(positions=torch.zeros(2, dtype=I32)), ValueError), (dict(slots=torch.zeros(6, dtype=I32)[::2]), ValueError),
    (dict(slots=None), TypeError), (dict(), ValueError),   # all well, but on the host
])
def test_rotary_append_refuses(monkeypatch, change, err):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    args = dict(qkv=torch.zeros(3, 256, dtype=BF), q_out=torch.zeros(3, 128, dtype=BF), positions=torch.zeros(3, dtype=I32),
                slots=torch.zeros(3, dtype=I32))
    args.update(change)
    rot = _object(rx.Rotary, device=0, rot_dim=32, interleaved=False)
    with pytest.raises(err):
        rx.rotary_append(rot, args["qkv"], 4, args["positions"], args["slots"], args["q_out"], _cpu_cache())


@pytest.mark.parametrize("change,err", [
    (dict(q=torch.zeros(3, 128)), TypeError), (dict(q=torch.zeros(3, 64, dtype=BF)), ValueError),
    (dict(out=torch.zeros(4, 128, dtype=BF)), ValueError), (dict(block_table=torch.zeros(2, 4, dtype=torch.int64)), TypeError),
    (dict(block_table=torch.zeros(1, 4, dtype=I32)), ValueError), (dict(block_table=torch.zeros(8, dtype=I32)), ValueError),
    (dict(block_table=torch.zeros(4, 2, dtype=I32).t()), ValueError), (dict(seq_lens=torch.zeros(1, dtype=I32)), ValueError),
    (dict(query_start=torch.zeros(0, dtype=I32)), ValueError), (dict(query_start=[0, 1, 3]), TypeError), (dict(), ValueError),
])
def test_paged_attention_refuses(monkeypatch, change, err):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    args = dict(q=torch.zeros(3, 128, dtype=BF), out=torch.zeros(3, 128, dtype=BF), block_table=torch.zeros(2, 4, dtype=I32),
                seq_lens=torch.zeros(2, dtype=I32), query_start=torch.zeros(3, dtype=I32))
    args.update(change)
    att = _object(rx.Attention, device=0, num_q_heads=4, num_kv_heads=2, head_dim=32)
    with pytest.raises(err):
        rx.paged_attention(att, args["q"], _cpu_cache(), args["block_table"], args["seq_lens"], args["query_start"], args["out"])


@pytest.mark.parametrize("change,err", [
    (dict(past=torch.zeros(3, dtype=torch.int64)), TypeError), (dict(new=torch.zeros(2, dtype=I32)), ValueError),
    (dict(new=torch.zeros(4, dtype=I32)), ValueError), (dict(tokens=9), ValueError), (dict(tokens=-1), ValueError),
    (dict(cursor=torch.zeros(2, dtype=I32)), ValueError), (dict(ring=torch.zeros(0, dtype=I32)), ValueError),
    (dict(table=torch.zeros(2, 4, dtype=I32)), ValueError), (dict(past=torch.zeros(5, dtype=I32), new=torch.zeros(5, dtype=I32)), ValueError),
    (dict(), ValueError),
])
def test_page_plan_refuses(monkeypatch, change, err):
    monkeypatch.setattr(rx.kv, "lib", _NoCalls())
    a = dict(past=torch.zeros(3, dtype=I32), new=torch.zeros(3, dtype=I32), tokens=8, ring=torch.zeros(8, dtype=I32),
             cursor=torch.zeros(4, dtype=I32), table=torch.zeros(3, 4, dtype=I32))
    a.update(change)
    plan = _object(rx.PagePlan, device=0, max_seqs=4, max_tokens=8, _out=[0] * 5)
    with pytest.raises(err):
        rx.page_plan(plan, a["past"], a["new"], a["tokens"], a["ring"], a["cursor"], a["table"], 16)


# ------------------------------------------------------------------------- the oracle
def test_oracle_plan_by_hand():
    """Pages of 16; ring of 6 from place 4: ids 9 (at 4), 8 (at 5), 7 (at 0) free."""
    ring = [7, -1, -1, -1, 9, 8]
    table = [[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, -1, -1]]
    out, tab, rg, cur = KO.page_plan([32, 5, 20], [2, 3, -1], table, 4, [x % 10 for x in ring] and ring, [4, 3], 16, 6)
    # request 0 needs one page (id 9, but 9 >= 6 places: not a page of this cache), request 1 none
    assert out["query_start"] == [0, 2, 5, 5] and out["seq_lens"] == [34, 8, 0]
    assert out["positions"] == [32, 33, 5, 6, 7, 0]
    assert out["slots"] == [-1, -1, 37, 38, 39, -1]
    assert tab[0].tolist() == [0, 1, -1, -1] and cur == [5, 4]
    assert rg.tolist() == [7, 3, 4, -1, 9, 8]
    assert out["meta"] == [5, 1, 2, 0, 1, 4, 0, 0]


def test_oracle_attention_by_hand():
    keys = np.zeros((2, 16, 1, 2))
    vals = np.zeros((2, 16, 1, 2))
    keys[1, 0, 0], keys[1, 1, 0] = [1, 0], [0, 1]
    vals[1, 0, 0], vals[1, 1, 0] = [1, 2], [3, 4]
    q = np.array([[[math_ln3, 0.0]]])
    out, lse, mass, smax = KO.attend(q, keys, vals, [[1]], [2], [0, 1], 16, 1.0)
    np.testing.assert_allclose(out[0, 0], [0.75 * 1 + 0.25 * 3, 0.75 * 2 + 0.25 * 4], rtol=1e-15)   # weights 3 : 1
    np.testing.assert_allclose(lse[0, 0], np.log(4.0), rtol=1e-15)
    out, lse, _, _ = KO.attend(q, keys, vals, [[1]], [2], [0, 1], 16, 1.0, window=1)
    np.testing.assert_allclose(out[0, 0], [3, 4])
    out, lse, _, _ = KO.attend(q, keys, vals, [[-1]], [2], [0, 1], 16, 1.0)
    assert not out.any() and lse[0, 0] == -np.inf


math_ln3 = float(np.log(3.0))


def test_oracle_e4m3_matches_torch():
    x = np.concatenate([np.random.default_rng(0).normal(size=4000) * s for s in (1e-3, 0.05, 1.0, 60.0, 400.0)])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(KO.e4m3_round(x.astype(np.float64)), want)
