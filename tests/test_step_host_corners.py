"""What can be told on the host about the serving step's operators at the edges of what their documentation allows (CPU only)."""
import ctypes as C
import glob
import os
import re
import types

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WAIT = "grid_dependency_wait();"


def kernels():
    """Each kernel's source: (file, name, body)."""
    for path in sorted(glob.glob(os.path.join(ROOT, "block_sparse_top_msa_gb300", "csrc", "*.cu"))):
        text = open(path).read()
        for m in re.finditer(r"__global__.*?\b(\w+_kernel)\((.*?)\n}\n", text, re.S):
            yield os.path.basename(path), m.group(1), re.sub(r"//[^\n]*", "", m.group(2))


def enclosing_block(text, at):
    """What stands in the innermost braces around a place, before it."""
    depth = 0
    for i in range(at - 1, -1, -1):
        depth += (text[i] == "}") - (text[i] == "{")
        if depth < 0:
            return text[i:at]
    return text[:at]


def test_dependent_kernels_wait_on_every_path():
    """A grid launched to begin under the tail of the one before it is ordered by its wait alone, and the grid after it by its end: a
    path that leaves before the wait orders nothing."""
    waiting = {name: (file, body) for file, name, body in kernels() if WAIT in body}
    launched = set()
    for path in glob.glob(os.path.join(ROOT, "block_sparse_top_msa_gb300", "csrc", "*.cu")):
        text = open(path).read()
        launched |= set(re.findall(r"(?:launch_dependent|launch_pdl)\(\s*(?:a\.interleaved \? )?(\w+_kernel)\b", text))
        launched |= set(re.findall(r"cudaLaunchKernelEx\(&cfg, (\w+_kernel)\b", text))
    assert len(launched) >= 14 and launched <= set(waiting), launched - set(waiting)
    for name in sorted(launched):
        file, body = waiting[name]
        # The wait that every thread comes to; the attention kernel has another for launches that wait late, in the work counter's claim.
        m = re.search(r"^  (?:if \(!a\.wait_late\) )?grid_dependency_wait\(\);", body, re.M)
        assert m, (file, name)
        before = body[: m.start()]
        for r in re.finditer(r"return;", before):
            assert WAIT in enclosing_block(before, r.start()), (file, name, before[max(0, r.start() - 200) : r.end()])


class Grid(C.Structure):
    _fields_ = [("q_blocks", C.c_int), ("k_blocks", C.c_int)]


def test_the_gradient_has_blocks_for_both_sides():
    """However unlike the head counts: a side with tokens has a block, and the two no more than the workspace has rows for."""
    import block_sparse_top_msa_gb300 as msa
    msa.build()
    L = msa.lib()
    grid = getattr(L, "_ZN3msa13rope_bwd_gridExii")  # msa::rope_bwd_grid(long long, int, int)
    grid.restype, grid.argtypes = Grid, [C.c_longlong, C.c_int, C.c_int]
    for tokens in (1, 12, 100, 1000, 65536, 10**6):
        for hq in (1, 4, 5, 64, 1300, 2048, 8192):
            for hkv in (1, 2, 8, 1300, 2048, 8192):
                g = grid(tokens, hq, hkv)
                assert g.q_blocks >= 1 and g.k_blocks >= 1 and g.q_blocks + g.k_blocks <= 304, (tokens, hq, hkv, g.q_blocks, g.k_blocks)
                assert L.msa_qk_norm_rope_bwd_workspace_size(tokens, hq, hkv) >= (g.q_blocks + g.k_blocks) * 512
    g = grid(0, 64, 8)
    assert g.q_blocks == 0 and g.k_blocks == 0


def test_a_prepared_tree_call_runs_on_its_own_device(monkeypatch):
    """Tensors on another device than the current one: that device is made current and its stream taken."""
    import torch

    import block_sparse_top_msa_gb300 as msa
    at, launched = [0], []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            at.append(self.device.index)

        def __exit__(self, *a):
            at.pop()

    class Library:
        msa_sparse_attention_plan_free = staticmethod(lambda plan: None)

        @staticmethod
        def msa_sparse_attention_run(plan, stream):
            launched.append((at[-1], stream.value))
            return 0

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=100 + at[-1]))
    r = msa.TreeAttentionRunner.__new__(msa.TreeAttentionRunner)
    r.out, r.lse, r._lib, r._plan = types.SimpleNamespace(device=torch.device("cuda", 3)), None, Library, C.c_void_p(1)
    assert r.run() is r.out
    r.run(stream=77)
    assert launched == [(3, 103), (3, 77)] and at == [0]


def test_pools_that_share_a_part_of_their_memory_are_refused():
    """In ascending order and in any other; the same pool twice is refused where rows move, and copied twice elsewhere."""
    import block_sparse_top_msa_gb300 as msa
    msa.build()
    L = msa.lib()
    P, INVALID = C.c_void_p(0x10000), 1
    pages, page = 4, 1 << 20

    def calls(*at):
        pools, n = (C.c_void_p * len(at))(*at), len(at)
        yield L.msa_cache_fork(pools, n, page, P, 4, 8, P, P, pages, P, P, 1, C.c_void_p(0x20000), P, 1 << 20, None)
        yield L.msa_cache_copy_pages(pools, n, page, pages, P, P, 1, None)
        yield L.msa_cache_accept(pools, n, 256, page // 256 // 128, P, 4, pages, 1, P, P, P, P, 3, C.c_void_p(0x20000), None)

    base = 1 << 32
    for at in ([0, 3], [3, 0], [0, 4, 8, 11], [8, 0, 4, 5], [0, 4, 3], [4, 4, 7]):
        assert list(calls(*[base + x * page for x in at])) == [INVALID] * 3, at
    assert list(calls(base, base + 4 * page - 16)) == [INVALID] * 3


def test_results_in_the_place_of_what_is_read_are_refused():
    import block_sparse_top_msa_gb300 as msa
    msa.build()
    L = msa.lib()
    P, Q, R, INVALID = C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x30000), 1
    pools = (C.c_void_p * 1)(1 << 32)
    for status in (P, Q):
        assert L.msa_cache_extend(R, 4, 8, R, R, 10, P, Q, 1, status, R, 1 << 20, None) == INVALID
        assert L.msa_cache_fork(pools, 1, 64, R, 4, 8, R, R, 10, P, Q, 1, status, R, 1 << 20, None) == INVALID
    for out in (P, Q):
        assert L.msa_cache_accept(pools, 1, 256, 2, R, 4, 10, 1, P, R, R, Q, 3, out, None) == INVALID
    tree = lambda out: L.msa_tree_attention(P, 0, Q, Q, 0, R, 4, R, R, 1, R, 4, 4, R, 1, 5, 8, 2, 128, 5, 0.0, out, None, R, 1 << 30, None)
    assert tree(P) == INVALID
