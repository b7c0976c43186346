"""Host-side checks of the decode-step entry points (include/gbfuse_decode.h):
exports, argument validation of the C ABI with addresses that are never read,
and the Python binding's operand checks.  No kernel is launched."""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

from conftest import ROOT

F = 1 << 32           # fake, 16-byte aligned addresses, far apart


def A(i, off=0):
    return ctypes.c_void_p(F * (i + 1) + off)


@pytest.fixture(scope="module")
def gbf():
    import fusion_add_rmsnorm_gb300 as g
    return g


def last(gbf):
    return gbf.raw().gbf_last_error().decode()


def test_decode_header_and_exports(gbf):
    text = open(os.path.join(ROOT, "include", "gbfuse_decode.h")).read()
    declared = set(re.findall(r"GBF_API\s+[\w\s\*]+?\b(gbfd_\w+)\s*\(", text))
    out = subprocess.run(["nm", "-D", "--defined-only", gbf.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (gbfd_\w+)", out)) == declared == set(gbf.EXPORTED_DECODE)


def call(fn, names, over):
    args = [over.pop(n, d) for n, d in names]
    assert not over, over
    return fn(*args)


def test_paged_slots_validation(gbf):
    names = lambda: [("ctx", A(0)), ("new", A(1)), ("batch", 4), ("table", A(2)), ("stride", 8), ("width", 8),   # noqa
                     ("bs", 16), ("free", A(3)), ("ring", A(4)), ("blocks", 64), ("seq", A(5)), ("ring_out", A(6)),
                     ("slots", A(7)), ("pos", A(8)), ("tokens", 4), ("start", A(9)), ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfd_paged_slots, names(), k)                                  # noqa: E731
    assert f(batch=0) == gbf.OK
    for bad in (dict(batch=-1), dict(bs=0), dict(tokens=-1), dict(blocks=0), dict(width=9), dict(width=-1)):
        assert f(**bad) == gbf.EINVAL, bad
    assert f(batch=8193) == gbf.EUNSUPPORTED and "8192" in last(gbf)
    assert f(blocks=1 << 30, bs=2) == gbf.EUNSUPPORTED
    assert f(tokens=1 << 31) == gbf.EUNSUPPORTED
    for p in ("ctx", "new", "table", "free", "ring", "seq", "ring_out", "slots", "pos"):
        assert f(**{p: None}) == gbf.EINVAL, p
    assert f(seq=A(1)) == gbf.EINVAL                   # an output on the new lengths
    assert f(seq=A(0, 4)) == gbf.EINVAL                # a shifted overlap is no in-place update
    assert f(ring_out=A(4, 4)) == gbf.EINVAL
    assert f(slots=A(8, 8)) == gbf.EINVAL and "outputs overlap" in last(gbf)
    assert f(start=A(2, 3 * 32)) == gbf.EINVAL         # inside the last table row
    assert f(start=A(5, 12)) == gbf.EINVAL


def test_paged_attention_validation(gbf):
    names = lambda: [("q", A(0)), ("k", A(1)), ("v", A(2)), ("rows", 256), ("table", A(3)), ("stride", 8),   # noqa: E731
                     ("width", 8), ("bs", 16), ("lens", A(4)), ("batch", 4), ("hq", 8), ("hkv", 2), ("d", 128),
                     ("scale", 0.1), ("window", 0), ("out", A(5)), ("out_scale", 0.0), ("lse", A(6)), ("ws", A(7)),
                     ("ws_bytes", 1 << 24), ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfd_paged_attention, names(), k)                              # noqa: E731
    inf, nan = float("inf"), float("nan")
    assert f(batch=0) == gbf.OK
    for bad in (dict(batch=-1), dict(hq=0), dict(hkv=3), dict(bs=0), dict(width=9), dict(window=-1), dict(rows=-1),
                dict(scale=0.0), dict(scale=inf), dict(scale=nan), dict(out_scale=-1.0), dict(out_scale=nan),
                dict(out_scale=1e-40), dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None),
                dict(out=None), dict(ws=None), dict(ws_bytes=1000)):
        assert f(**bad) == gbf.EINVAL, bad
    for bad in (dict(d=72), dict(d=272), dict(rows=1 << 31), dict(batch=1 << 29), dict(hq=8192, hkv=2)):
        assert f(**bad) == gbf.EUNSUPPORTED, bad
    for p in ("q", "k", "v", "out", "ws"):
        assert f(**{p: A(9, 8)}) == gbf.EALIGN, p
    for p in ("q", "k", "v", "table", "lens"):
        i = {"q": 0, "k": 1, "v": 2, "table": 3, "lens": 4}[p]
        assert f(out=A(i)) == gbf.EINVAL and f(lse=A(i)) == gbf.EINVAL and f(ws=A(i)) == gbf.EINVAL, p
    assert f(lse=A(5, 64)) == gbf.EINVAL and f(ws=A(5)) == gbf.EINVAL
    w = gbf.raw().gbfd_paged_attention_workspace
    assert w(8, 2, 128) > 0 and w(8, 3, 128) == 0 and w(8, 2, 100) == 0 and w(8, 2, 512) == 0 and w(0, 0, 0) == 0
    assert f(ws_bytes=w(8, 2, 128) - 1) == gbf.EINVAL and "needs" in last(gbf)


def test_sample_tokens_validation(gbf):
    names = lambda: [("logits", A(0)), ("f32", 0), ("batch", 4), ("vocab", 1000), ("stride", 1000), ("u", A(1)),   # noqa
                     ("t", A(2)), ("k", A(3)), ("p", A(4)), ("mp", A(5)), ("tokens", A(6)), ("logprob", A(7)),
                     ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfd_sample_tokens, names(), k)                                # noqa: E731
    assert f(batch=0) == gbf.OK
    for bad in (dict(batch=-1), dict(vocab=0), dict(f32=2), dict(stride=999), dict(logits=None), dict(u=None),
                dict(tokens=None), dict(tokens=A(0, 16)), dict(logprob=A(6, 4)), dict(logprob=A(5)), dict(tokens=A(3))):
        assert f(**bad) == gbf.EINVAL, bad
    assert f(vocab=(1 << 20) + 1, stride=1 << 21) == gbf.EUNSUPPORTED
    assert f(logits=A(0, 8)) == gbf.EALIGN


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)     # noqa: E731
u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)        # noqa: E731
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)       # noqa: E731
f32 = lambda *s: torch.zeros(*s, dtype=torch.float32)     # noqa: E731


def raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_paged_slots_operands(gbf):
    good = dict(ctx_lens=i32(3), new_lens=i32(3), block_table=i32(3, 4), free_ring=i32(16), ring=i32(2), block_size=16,
                seq_lens=i32(3), ring_out=i32(2), slots=i32(5), pos=i32(5), start=i32(4))
    for name, t in (("new_lens", i32(2)), ("seq_lens", i32(4)), ("ring", i32(3)), ("ring_out", i32(1)), ("pos", i32(4)),
                    ("start", i32(3)), ("block_table", i32(2, 4)), ("block_table", i32(12)),
                    ("block_table", i32(4, 3).t())):
        raises(name, gbf.paged_slots, **{**good, name: t})
    raises("CUDA device", gbf.paged_slots, **good)
    raises("CUDA device", gbf.paged_slots, **{**good, "block_table": i32(3, 9)[:, 2:6]})


def test_paged_attention_operands(gbf):
    good = dict(q=bf(2, 8, 64), k_cache=bf(32, 2, 64), v_cache=bf(32, 2, 64), block_table=i32(2, 2), seq_lens=i32(2),
                block_size=16, out=bf(2, 8, 64), workspace=u8(1 << 22), lse=f32(2, 8))
    for name, t in (("q", bf(16, 64)), ("k_cache", bf(32, 2, 32)), ("k_cache", bf(32, 128)), ("v_cache", bf(31, 2, 64)),
                    ("seq_lens", i32(3)), ("out", bf(2, 8, 32)), ("lse", f32(2, 4)), ("block_table", i32(3, 2))):
        raises(name, gbf.paged_attention, **{**good, name: t})
    raises("out_scale", gbf.paged_attention, **{**good, "out_scale": 0.0})
    raises("CUDA device", gbf.paged_attention, **good)
    raises("not supported", gbf.paged_attention_workspace, 8, 3, 64)


def test_sample_tokens_operands(gbf):
    good = dict(logits=bf(3, 40), uniform=f32(3), tokens=i32(3), temperature=f32(3), top_k=i32(3), top_p=f32(3),
                min_p=f32(3), logprob=f32(3))
    for name in ("uniform", "temperature", "top_p", "min_p", "logprob"):
        raises(name, gbf.sample_tokens, **{**good, name: f32(4)})
    for name in ("tokens", "top_k"):
        raises(name, gbf.sample_tokens, **{**good, name: i32(2)})
    raises("logits", gbf.sample_tokens, **{**good, "logits": bf(40, 3).t()})
    raises("logits", gbf.sample_tokens, **{**good, "logits": bf(120)})
    raises("CUDA device", gbf.sample_tokens, **good)
    with pytest.raises(TypeError, match="logits"):
        gbf.sample_tokens(**{**good, "logits": torch.zeros(3, 40, dtype=torch.float16)})


def test_compiled_wrappers_arguments(gbf):
    slots = dict(ctx_lens=i32(3), new_lens=i32(3), block_table=i32(3, 4), free_ring=i32(16), ring=i32(2), block_size=16,
                 seq_lens=i32(3), ring_out=i32(2), slots=i32(5), pos=i32(5))
    attn = dict(q=bf(2, 8, 64), k_cache=bf(32, 2, 64), v_cache=bf(32, 2, 64), block_table=i32(2, 2), seq_lens=i32(2),
                block_size=16, out=bf(2, 8, 64), workspace=u8(1 << 22))
    draw = dict(logits=bf(3, 40), uniform=f32(3), tokens=i32(3))
    for fn, good in ((gbf.paged_slots, slots), (gbf.paged_attention, attn), (gbf.sample_tokens, draw)):
        raises("CUDA device", fn, *good.values())                       # by position, the optional ones left out
        for name in good:
            with pytest.raises(TypeError, match=name):                  # a required argument left out
                fn(**{k: v for k, v in good.items() if k != name})
            with pytest.raises(TypeError, match=name):                  # not what the argument takes
                fn(**{**good, name: "x"})
        first = next(iter(good))
        with pytest.raises(TypeError, match=first):
            fn(*good.values(), **{first: good[first]})                  # given twice
        with pytest.raises(TypeError, match="blocks"):
            fn(**good, blocks=1)                                        # no such argument
        with pytest.raises(TypeError, match="at most"):
            fn(*[None] * 20)
    for name in ("ctx_lens", "block_table", "slots", "free_ring"):
        with pytest.raises(TypeError, match=name):
            gbf.paged_slots(**{**slots, name: slots[name].long()})
    with pytest.raises(TypeError, match="block_size"):
        gbf.paged_slots(**{**slots, "block_size": 16.0})
    raises("block_size", gbf.paged_slots, **{**slots, "block_size": 1 << 33})
    # an out_scale that is 0 in float32 would ask for bf16 output, twice the bytes that `out` holds
    for bad in (1e-60, -1.0, float("nan")):
        raises("out_scale", gbf.paged_attention, **{**attn, "out": u8(2, 8, 64), "out_scale": bad})
    with pytest.raises(TypeError, match="out"):
        gbf.paged_attention(**{**attn, "out_scale": 1.0})


def test_clusters_have_started_before_they_write_to_each_other():
    """Shared memory of another CTA may be touched only once that CTA is known to run, which nothing shows from
    outside: in the sampling kernel all ranks arrive at its start, and wait before the first exchange."""
    text = open(os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "csrc", "sample_tokens.cu")).read()
    kernel = text[text.index("sample_kernel(const SampleArgs a) {"):]
    arrive, wait = kernel.find("cluster.barrier_arrive();"), kernel.find("cluster.barrier_wait();")
    first = min(kernel.index(f"s.{f}(") for f in ("exchange", "offer", "of", "find_bins", "close_lists"))
    assert 0 <= arrive < kernel.index("pdl_wait();") < wait < first


def test_the_join_starts_behind_the_lengths():
    """paged_attention's join reads the lengths before its own wait.  That holds as long as every CTA of the kernel in
    front waits first of all and lets the join begin only then, and the join reads them from L2."""
    text = open(os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "csrc", "paged_attention.cu")).read()
    text = re.sub(r"//[^\n]*", "", text)
    main = text[text.index("    paged_attention_kernel(const PagedAttnArgs a) {"):]
    wait, begin = main.index("pdl_wait();"), main.index("pdl_launch_dependents();")
    assert wait < begin < min(main.index(s) for s in ("return", "a.lens", "a.table", "locate<"))
    join = text[text.index("paged_attention_join_kernel(const PagedAttnArgs a) {"):]
    early = join[:join.index("  pdl_wait();\n")]
    assert "locate<128, true>(" in early and "request_of<true>(" in early
    assert not re.search(r"a\.(lens|ws|table|q|k|v|out|lse)\b", early)


def test_paged_attention_batches_the_split_can_count(gbf):
    """The scan over the lengths counts requests in 32 bits and steps past the end of them: 2^30 at most."""
    names = lambda: [("q", A(0)), ("k", A(100)), ("v", A(200)), ("rows", 256), ("table", A(300)), ("stride", 1),   # noqa
                     ("width", 1), ("bs", 16), ("lens", A(400)), ("batch", 4), ("hq", 1), ("hkv", 1), ("d", 16),
                     ("scale", 0.1), ("window", 0), ("out", A(500)), ("out_scale", 0.0), ("lse", None), ("ws", A(600)),
                     ("ws_bytes", 0), ("stream", None)]
    f = lambda **k: call(gbf.raw().gbfd_paged_attention, names(), k)                              # noqa: E731
    for batch in ((1 << 30) + 1, (1 << 31) - 1, 1 << 31, 1 << 62):
        assert f(batch=batch) == gbf.EUNSUPPORTED and "2^30" in last(gbf), batch
    assert f(batch=1 << 30) == gbf.EINVAL and "workspace" in last(gbf)


def copy_of_the_package(tmp_path, *built):
    here = tmp_path / "fusion_add_rmsnorm_gb300"
    here.mkdir()
    for name in ("__init__.py", "libgbfuse.so", *built):
        (here / name).symlink_to(os.path.join(ROOT, "fusion_add_rmsnorm_gb300", name))
    return str(tmp_path)


WITHOUT = """
import torch
import fusion_add_rmsnorm_gb300 as gbf
assert gbf.__file__.startswith({path!r}), gbf.__file__
assert gbf.version() > 0 and gbf.paged_attention_workspace(8, 2, 64) > 0
f = lambda *s: torch.zeros(*s)
try:
    gbf.bn_fold(f(4, 8), f(4), f(4), f(4), f(4), f(4), 1e-5, f(4, 8), f(4))
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise SystemExit("bn_fold ran on the CPU")
for name in ("paged_slots", "paged_attention", "sample_tokens"):
    try:
        getattr(gbf, name)(1, stream=None)
    except ImportError as e:
        assert name in str(e) and "build.py" in str(e) and {why!r} in str(e), e
    else:
        raise SystemExit(name + " was there")
"""


def run_python(path, code):
    r = subprocess.run([sys.executable, "-c", code], cwd=path, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": path})
    assert r.returncode == 0, r.stderr[-2000:]


def test_without_the_extension_the_other_operators_are_there(tmp_path):
    path = copy_of_the_package(tmp_path)
    run_python(path, WITHOUT.format(path=path, why="decode_binding"))


def test_the_extension_names_its_python_and_torch(gbf, tmp_path):
    import sysconfig
    name = "decode_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(gbf._decode.__file__) == name and gbf._decode.built_for_torch == torch.__version__
    path = copy_of_the_package(tmp_path, name)
    other = "import torch; torch.__version__ = '1.0.other'\n" + WITHOUT.format(path=path, why="this is torch 1.0.other")
    run_python(path, other)


def test_an_extension_that_names_no_torch_is_not_used(tmp_path):
    """As builds before the version was noted left it."""
    path = copy_of_the_package(tmp_path)
    (tmp_path / "fusion_add_rmsnorm_gb300" / "decode_binding.py").write_text("paged_slots = print\n")
    run_python(path, WITHOUT.format(path=path, why="unknown version"))
