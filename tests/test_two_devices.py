"""Calls on two devices of one process, over a stand-in for the CUDA runtime: the library's
own objects linked against a few functions that count launches and, as the runtime does,
refuse one whose dynamic shared memory the current device has not been asked for.  Nothing
is computed and no GPU is used."""

import ctypes
import os
import subprocess

import pytest

from invariant_decode_attention_gb300 import build as B

RUNTIME = r"""
#include <cstdint>
#include <cstring>
#include <map>
#include <utility>

#include <cuda_runtime_api.h>

static int g_device, g_launches, g_failures;
static std::map<std::pair<int, const void*>, int> g_smem;
static char g_symbol[1 << 12];

static int encode(...) { return 0; }

extern "C" {
void stand_in_device(int device, int failures) { g_device = device; g_failures = failures; }
int stand_in_launches() { return g_launches; }

cudaError_t cudaGetDevice(int* d) { *d = g_device; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int bytes) {
  if (g_failures > 0) { --g_failures; return cudaErrorUnknown; }
  g_smem[{g_device, f}] = bytes;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *f = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = g_symbol; return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto at = g_smem.find({g_device, f});
  const size_t allowed = at == g_smem.end() ? 48 * 1024 : at->second;
  if (c->dynamicSmemBytes > allowed) return cudaErrorInvalidValue;
  ++g_launches;
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = 1;
  return cudaSuccess;
}
// what compiled sources call to make their kernels known
void** __cudaRegisterFatBinary(void*) { static void* handle[1]; return handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(...) {}
void __cudaRegisterVar(...) {}
int __cudaGetKernel(...) { return 0; }
int __cudaLaunchKernel(...) { ++g_launches; return 0; }
int __cudaPopCallConfiguration(...) { return 0; }
unsigned __cudaPushCallConfiguration(...) { return 0; }
}
"""


@pytest.fixture(scope="module")
def api(tmp_path_factory):
    from invariant_decode_attention_gb300 import api as _api
    folder = tmp_path_factory.mktemp("runtime")
    source, path = folder / "runtime.cc", folder / "libstandin.so"
    source.write_text(RUNTIME)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.nvcc()))), "include")
    objects = [os.path.join(B.OBJ_DIR, f + ".o") for f in sorted(os.listdir(B.CSRC)) if f.endswith(".cu")]
    if not all(os.path.exists(o) for o in objects):
        B.build()
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wl,-Bsymbolic", "-I", include, str(source),
                    *objects, "-o", str(path)], check=True)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(_api, "LIB_PATH", str(path))
        m.setattr(_api, "_LIB", None)
        _api.lib().stand_in_launches.restype = ctypes.c_int
        yield _api


def tree(api, kv, D, T, group):
    p = api.problem(batch=2, num_q_heads=2 * group, num_kv_heads=2, head_dim_qk=D, layout="paged", scale=0.1,
                    page_size=16, width=64, num_blocks=200, kv_dtype=kv)
    args = api._TREE.pack(T, 0, 0, 0, 0, 1 << 20, 1 << 28, 1 << 29, 1 << 23, 1 << 24, 1 << 26, 1 << 25, 0, 1 << 30,
                          api.tree_workspace_bytes(p, T))
    return api.lib().decode_attn_tree(ctypes.addressof(p), args, None)


def forward(api, kv, D, group, page=16, latent=False, extra=False):
    H = 1 if latent else 2
    p = api.problem(batch=2, num_q_heads=H * group, num_kv_heads=H, head_dim_qk=D, head_dim_v=512 if latent else D,
                    layout="paged" if page else "indexed", scale=0.1, page_size=page, width=64, num_blocks=200,
                    kv_dtype=kv, shared_latent=latent, extra_width=8 if extra else 0, extra_num_blocks=9 if extra else 0)
    ref, v, table, lengths, more = ctypes.byref(p), 0 if latent else 1 << 22, 1 << 23, 1 << 24, 1 << 25
    rest = (1 << 30, api.workspace_bytes(p), 1 << 26, 1 << 28, None)
    if not extra:
        return api.lib().decode_attn_forward(ref, api.INVARIANT, 1 << 20, 1 << 21, v, table, lengths, *rest)
    return api.lib().decode_attn_forward_extra(ref, api.INVARIANT, 1 << 20, 1 << 21, v, table, lengths, more,
                                               0 if latent else more, more, more, *rest)


def matmul(api):
    n, N, K = 40, 256, 2048
    return api.lib().nvfp4_mm(1 << 20, 1, 1 << 21, 1 << 22, 1.0, n, N, K, 1 << 23, 0, 1 << 30,
                              api.lib().nvfp4_mm_workspace_bytes(n, N, K), None)


# (T, query heads a KV head): every width of the kernel for few rows, and the tiles of 128
CALLS = [(f"tree kv{kv} D{D} T{T} group {group}", lambda api, a=(kv, D, T, group): tree(api, *a))
         for kv in (0, 1, 2) for D in (64, 128) for T, group in ((1, 4), (4, 4), (6, 4), (8, 4), (16, 4))]
CALLS += [(f"attention kv{kv} D{D} group {group} page {page}", lambda api, a=(kv, D, group, page): forward(api, *a))
          for kv in (0, 1, 2) for D in (64, 128) for group in (1, 2, 4, 8) for page in (16, 64)]
CALLS += [(f"attention kv{kv} group {group}", lambda api, a=(kv, 128, group): forward(api, *a))
          for kv in (0, 1, 2) for group in (16, 32, 64, 128)]
CALLS += [(f"latent attention kv{kv}", lambda api, kv=kv: forward(api, kv, 576, 64, latent=True)) for kv in (0, 1)]
CALLS += [(f"attention of two sources, group {group}", lambda api, group=group: forward(api, 0, 128, group, 0, extra=True))
          for group in (1, 2, 4)]
CALLS += [("matmul", matmul)]


@pytest.mark.parametrize("call", [c for _, c in CALLS], ids=[n for n, _ in CALLS])
def test_each_device_is_asked(api, call):
    runtime = api.lib()
    for device in (0, 1, 0, 2):
        runtime.stand_in_device(device, 0)
        before = runtime.stand_in_launches()
        assert call(api) == api.OK
        assert runtime.stand_in_launches() > before


@pytest.mark.parametrize("call", [c for _, c in CALLS], ids=[n for n, _ in CALLS])
def test_a_failure_is_not_kept(api, call):
    runtime = api.lib()
    runtime.stand_in_device(5, 1 << 20)
    assert call(api) == api.ERR_CUDA
    runtime.stand_in_device(5, 0)
    assert call(api) == api.OK
