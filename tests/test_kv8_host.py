"""Refusals of the 8-bit paged cache's entry points (no GPU): every bad argument is answered
before anything is enqueued, and the binding refuses tensors it cannot hand on."""
import pytest
import torch

FAKE = 1 << 20  # a 16-byte-aligned non-null address; validation answers before any use

INVALID, UNSUPPORTED, WORKSPACE, CUDA = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    from exact_tiled_attention_20_gb300 import _lib, build

    build.build_library()
    return _lib._load_fp8()


APPEND = dict(k_new=FAKE, v_new=FAKE, k_stride=1024, v_stride=1024, cu=None, table=FAKE, lens=FAKE, k=FAKE, v=FAKE,
              ks=FAKE, vs=FAKE, B=2, total=4, Hkv=8, D=128, num_pages=9, page=16, max_pages=4, dtype=0, stream=None)
READ = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, starts=None, cu=FAKE, ko=FAKE, vo=FAKE, B=2, total=4, Hkv=8,
            D=128, num_pages=9, page=16, max_pages=4, dtype=0, stream=None)
DECODE = dict(q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, table=FAKE, lens=FAKE, o=FAKE, lse=None, B=2, Sq=1, Hq=16,
              Hkv=8, D=128, num_pages=9, page=16, max_pages=4, scale=0.1, causal=1, splits=4, ws=FAKE,
              ws_bytes=1 << 30, dtype=0, stream=None)

POOL = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
        (dict(table=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 4), INVALID),
        (dict(ks=FAKE + 1), INVALID), (dict(vs=FAKE + 8), INVALID), (dict(table=FAKE + 2), INVALID),
        (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(page=0), INVALID),
        (dict(page=-16), INVALID), (dict(max_pages=0), INVALID), (dict(page=24), UNSUPPORTED),
        (dict(page=1), UNSUPPORTED), (dict(D=80), UNSUPPORTED), (dict(D=0), UNSUPPORTED), (dict(D=512), UNSUPPORTED),
        (dict(dtype=2), UNSUPPORTED), (dict(B=1026), UNSUPPORTED),
        (dict(page=1 << 20, max_pages=1 << 11), UNSUPPORTED),
        (dict(page=16, max_pages=(1 << 27) - 1), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED)]


@pytest.mark.parametrize("change,code", POOL + [
    (dict(lens=None), INVALID), (dict(lens=FAKE + 2), INVALID), (dict(cu=FAKE + 1), INVALID),
    (dict(total=-1), INVALID), (dict(total=5), INVALID), (dict(k_new=None), INVALID), (dict(v_new=FAKE + 2), INVALID),
    (dict(k_stride=1016), INVALID), (dict(v_stride=1028), INVALID), (dict(k_stride=-1024), INVALID),
    (dict(total=1 << 29), UNSUPPORTED), (dict(total=0), 0), (dict(total=0, k_new=None, v_new=None), 0)])
def test_append_refuses(lib, change, code):
    assert lib.fa_kv_append_paged_fp8(*{**APPEND, **change}.values()) == code


@pytest.mark.parametrize("change,code", POOL + [
    (dict(cu=None), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(starts=FAKE + 1), INVALID), (dict(total=-1), INVALID),
    (dict(ko=None), INVALID), (dict(vo=FAKE + 2), INVALID), (dict(total=1 << 29), UNSUPPORTED),
    (dict(total=0, ko=None, vo=None), 0)])
def test_read_refuses(lib, change, code):
    assert lib.fa_kv_read_paged_fp8(*{**READ, **change}.values()) == code


@pytest.mark.parametrize("change,code", POOL + [
    (dict(q=None), INVALID), (dict(q=FAKE + 2), INVALID), (dict(o=None), INVALID), (dict(o=FAKE + 8), INVALID),
    (dict(lse=FAKE + 2), INVALID), (dict(lens=None), INVALID), (dict(Sq=0), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=12), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(Hq=136), UNSUPPORTED), (dict(Sq=9), UNSUPPORTED),
    (dict(B=1024, Hq=1 << 10, Hkv=1 << 10, max_pages=1 << 13), UNSUPPORTED)])
def test_decode_refuses(lib, change, code):
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **change}.values()) == code


def test_decode_refuses_partial_results_past_64_bits(lib):
    """2^23 rows and a count for which the bytes of the partial results pass 2^64 and come out small."""
    splits = -(-2 ** 39 // 257)
    assert 2 ** 23 * splits * 257 * 4 > 2 ** 64
    assert lib.fa_decode_workspace_bytes(1024, 1 << 13, 256, splits) < 1 << 40
    change = dict(B=1024, Hq=1 << 13, Hkv=1 << 13, D=256, splits=splits, ws_bytes=1 << 40)
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **change}.values()) == UNSUPPORTED


@pytest.mark.parametrize("change", [dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=16)])
def test_decode_refuses_a_bad_workspace(lib, change):
    if not torch.cuda.is_available():
        assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **change}.values()) == CUDA  # the SM count is not known
    else:
        assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **change}.values()) == WORKSPACE


def test_valid_calls_without_a_device_fail_loudly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.fa_kv_append_paged_fp8(*APPEND.values()) == CUDA
    assert lib.fa_kv_read_paged_fp8(*READ.values()) == CUDA
    assert lib.fa_decode_splitkv_paged_fp8(*DECODE.values()) == CUDA


def test_decode_takes_the_tables_that_append_and_read_take(lib):
    """Table capacities whose product with B passes 2^31 (the kernels count per pair, in 64-key units): up
    to the header's B * Hkv * (capacity / 64 + 8) < 2^31, not to 2^31 keys over the batch."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these arguments would be launched")
    wide = dict(B=2, Hkv=8, max_pages=(1 << 26) + 1)                        # 2^30 + 16 keys each
    assert lib.fa_kv_append_paged_fp8(*{**APPEND, **wide}.values()) == CUDA
    assert lib.fa_kv_read_paged_fp8(*{**READ, **wide}.values()) == CUDA
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **wide}.values()) == CUDA
    edge = dict(Hq=128, Hkv=128, max_pages=1 << 16, ws_bytes=1 << 50)         # 2^20 keys: 128 * (2^14 + 8) a sequence
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **edge, "B": 1023}.values()) == CUDA
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **edge, "B": 1024}.values()) == UNSUPPORTED


def test_decode_refuses_more_values_of_a_sequence_than_32_bits_count(lib):
    """8388608 rows of 256 values: an empty sequence's would be counted in 32 bits."""
    change = dict(B=1, Hq=1 << 23, Hkv=1 << 19, D=256, max_pages=1, splits=1)
    assert lib.fa_decode_splitkv_paged_fp8(*{**DECODE, **change}.values()) == UNSUPPORTED


def _cpu_pool(pages=3, Hkv=2, page=16, D=64, B=2):
    return (torch.zeros(pages, Hkv, page, D).to(torch.float8_e4m3fn), torch.zeros(pages, Hkv, page, D).to(torch.float8_e4m3fn),
            torch.zeros(pages, Hkv, page, dtype=torch.uint8), torch.zeros(pages, Hkv, page, dtype=torch.uint8),
            torch.zeros(B, 1, dtype=torch.int32))


def test_binding_rejects_cpu_tensors(lib):
    import exact_tiled_attention_20_gb300 as fa

    pool, lens = _cpu_pool(), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        fa.fa_kv_append_paged_fp8(x, x, *pool, lens)
    with pytest.raises(TypeError):
        fa.fa_kv_read_paged_fp8(*pool, torch.zeros(3, dtype=torch.int32), total=4)
    with pytest.raises(TypeError):
        fa.fa_decode_splitkv_paged_fp8(x, *pool, lens)


def test_import_needs_no_cuda_build_of_torch():
    """The package imports, and answers what needs no tensors, where torch lacks the names of its CUDA build."""
    import os
    import subprocess
    import sys

    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import exact_tiled_attention_20_gb300 as fa\n"
            "from exact_tiled_attention_20_gb300 import _lib\n"
            "assert fa.fa_decode_workspace_bytes(1, 1, 64, 1) > 0 and _lib._load_fp8() is not None\n"
            "try:\n"
            "    fa.fa_kv_read_paged_fp8(*[torch.zeros(1)] * 5, torch.zeros(2), total=1)\n"
            "except (TypeError, ValueError):\n"
            "    print('refused')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused"], r.stderr[-2000:]
