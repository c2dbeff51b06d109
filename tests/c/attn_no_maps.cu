// kvx_shared_attention over 4-bit pools where tensor maps cannot be made, on the host alone: the runtime's launches are
// stand-ins that note what they are given.  argv[1]: 0: the driver has no encoder; 1: its encoder refuses; 2: it encodes.
// Prints a line a call: status, launches, copies of the 4-bit kernel (AttnQ4Copies).
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <cuda.h>
#include <vector>

#include "kvx.h"
#include "kvx_attn.cuh"
#include "kvx_quant.cuh"

static int mode, launches;
static kvx::AttnParams seen;

static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                       const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return mode == 2 ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}

extern "C" cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned int, unsigned long long,
                                                        cudaDriverEntryPointQueryResult *r) {
  *f = mode == 0 ? nullptr : (void *)encode;
  *r = mode == 0 ? cudaDriverEntryPointSymbolNotFound : cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **args) {
  memcpy(&seen, args[0], sizeof(seen));
  ++launches;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }

int main(int, char **argv) {
  mode = atoi(argv[1]);
  const uint64_t at = 1ull << 40;  // an address that nothing reads
  for (int hnd = 0; hnd < 2; ++hnd)
    for (int D : {64, 128})
      for (int H : {1, 2, 3, 8, 12}) {
        const int64_t S = D / 8 * 5, slots = 1600;
        kvx_layout_desc d = {};
        d.num_layers = 2, d.kv_heads = H, d.head_dim = D, d.dtype = KVX_Q4, d.num_slots = slots;
        d.kind = hnd ? KVX_HND_PAGED : KVX_NHD, d.page_size = 16;
        d.base = (void *)at, d.plane_stride = slots * H * S;
        kvx_layout_t pool;
        if (kvx_layout_create(&d, &pool) != KVX_OK) return 2;
        kvx_attn_args a = {};
        a.layer = 1, a.q_dtype = KVX_BF16, a.q_heads = 4 * H, a.n_q = a.n_reqs = 3, a.page_size = 16;
        a.max_pages = a.table_stride = 8;
        a.q = (void *)(2 * at), a.out = (void *)(3 * at), a.tables = (const int32_t *)(4 * at);
        a.seq_lens = (const int32_t *)(5 * at);
        a.q_token_stride = a.out_token_stride = 4 * H * D, a.q_head_stride = a.out_head_stride = D;
        a.scale = a.k_scale = a.v_scale = 1.f;
        launches = 0;
        memset(&seen, 0, sizeof(seen));
        const kvx_status st = kvx_shared_attention(pool, &a, (void *)(6 * at), (size_t)1 << 32, (int32_t *)(7 * at), 0);
        printf("%s %d %d: %d %d %d\n", hnd ? "hnd" : "nhd", D, H, (int)st, launches, (int)seen.q4_copies);
        // where a stage's head vectors stand: apart from one another, and within the stage
        const int keys = 16 * (kvx::kAttnQ4Warps >> seen.slot_shift), stage = 2 * (128 * (int)S + (D == 128 ? 1024 : 512));
        std::vector<char> taken(stage, 0);
        for (int v = 0; v < 2; ++v)
          for (int k = 0; k < keys; ++k)
            for (int s = 0; s < seen.chunk; ++s) {
              const int64_t o = v * seen.q4_v_off + k / 16 * seen.q4_block_pitch + (s >> seen.q4_pair) * seen.q4_head_pitch +
                                (s & seen.q4_pair) * S + k % 16 * seen.q4_key_pitch;
              if (o < 0 || o + S > stage) return printf("a vector ends at %lld of %d\n", (long long)(o + S), stage), 1;
              for (int64_t i = o; i < o + S; ++i)
                if (taken[i]++) return printf("byte %lld of a stage twice\n", (long long)i), 1;
            }
        kvx_layout_destroy(pool);
      }
  return 0;
}
