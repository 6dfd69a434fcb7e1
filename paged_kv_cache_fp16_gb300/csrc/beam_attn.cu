// q4 attention of beams: checks, the plan and the entry points (the kernels are described in their header).
#include "beam_attn.cuh"

namespace kvq {
namespace beam {
namespace {

struct Plan {
  int nt;
  Line line[2];
  int64_t records, granules;
  size_t head_bytes() const {
    return (static_cast<size_t>(line[0].units + line[1].units + 1) * 8 + 15) / 16 * 16;
  }
};

Plan plan(int n_layers, int nseq, int beams, int H, int Hq, int D, int max_shared, int max_own) {
  Plan p;
  const int G = Hq / H;
  const int need = ((max_shared > 0 ? beams : 1) * G + 7) / 8;
  p.nt = std::min(need <= 1 ? 1 : need <= 2 ? 2 : 4, most_tiles(D));
  int64_t recs = 0, units = 0;
  p.granules = 0;
  for (int kind = 0; kind < 2; ++kind) {
    Line& L = p.line[kind];
    const int cols = (kind == 0 ? beams : 1) * G, tiles = (cols + 7) / 8;
    L.n = kind == 1 ? nseq : max_shared > 0 ? nseq / beams : 0;
    L.rep = n_layers * H;
    L.blocks = (tiles + p.nt - 1) / p.nt;
    L.weight = 2 + std::min(p.nt, tiles);
    L.most = L.n ? kMostBlocks / L.blocks + 1 : 0;
    L.solo = kind == 1 && cols <= 8 && static_cast<int64_t>(max_own) + kTile - 1 <= kGranule &&
             static_cast<int64_t>(L.n) * L.rep >= kSoloUnits;
    L.units = static_cast<int64_t>(L.n) * L.rep;
    L.first_unit = units;
    L.first_rec = recs;
    units += L.units;
    recs += L.blocks * (L.units + L.most);
    const int64_t tokens = kind == 0 ? max_shared : static_cast<int64_t>(max_own) + kTile - 1;
    p.granules += L.units * L.blocks * ((tokens + kGranule - 1) / kGranule);
  }
  p.records = recs;
  return p;
}

constexpr int kMostTokens = INT32_MAX - 64;   // of a sequence

bool bad_shape(int n_layers, int nseq, int beams, int H, int Hq, int D, int max_shared, int max_own) {
  return n_layers < 1 || n_layers > KVQ_MAX_TENSORS || nseq < 1 || nseq > KVQ_MAX_SEQS || beams < 1 ||
         beams > KVQ_MAX_BEAMS || nseq % beams != 0 || H < 1 || Hq < 1 || Hq % H != 0 ||
         Hq / H > 64 || (D != 64 && D != 128 && D != 256) || max_shared < 0 || max_own < 0 ||
         max_shared > kMostTokens || max_own > kMostTokens;
}

}  // namespace
}  // namespace beam
}  // namespace kvq

extern "C" size_t kvq_beam_attn_workspace(int n_layers, int nseq, int beams, int num_kv_heads,
                                          int num_q_heads, int head_dim, int max_shared, int max_own) {
  using namespace kvq::beam;
  if (bad_shape(n_layers, nseq, beams, num_kv_heads, num_q_heads, head_dim, max_shared, max_own)) return 0;
  const Plan p = plan(n_layers, nseq, beams, num_kv_heads, num_q_heads, head_dim, max_shared, max_own);
  return p.head_bytes() + static_cast<size_t>(p.records) * 8 * p.nt * (head_dim + 2) * 4;
}

extern "C" kvq_status kvq_beam_attn(kvq_dtype dtype, const kvq_pool* k_pools, const kvq_pool* v_pools,
                                    int n_layers, const uint16_t* q, int num_q_heads,
                                    const int32_t* page_table, int max_pages, const int32_t* seq_lens,
                                    const int32_t* shared_lens, int nseq, int beams, int max_shared,
                                    int max_own, float softmax_scale, uint16_t* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_err, kvq_stream_t stream) {
  using namespace kvq;
  using namespace kvq::beam;
  const char* fn = "kvq_beam_attn";
  if (dtype != KVQ_F16 && dtype != KVQ_BF16)
    return fail(KVQ_ERR_SHAPE, "%s: dtype %d is neither KVQ_F16 nor KVQ_BF16", fn,
                static_cast<int>(dtype));
  if (n_layers < 1 || n_layers > KVQ_MAX_TENSORS)
    return fail(KVQ_ERR_RANGE, "%s: n_layers %d not in [1, %d]", fn, n_layers, KVQ_MAX_TENSORS);
  kvq_status st = check_pools_uniform(k_pools, n_layers, fn);
  if (st != KVQ_OK) return st;
  st = check_pools_uniform(v_pools, n_layers, fn);
  if (st != KVQ_OK) return st;
  const kvq_pool& p0 = k_pools[0];
  const kvq_pool& p1 = v_pools[0];
  if (p0.bits != 4 || p1.bits != 4) return fail(KVQ_ERR_BITS, "%s: bits must be 4", fn);
  if (p1.num_heads != p0.num_heads || p1.head_dim != p0.head_dim || p1.page_size != p0.page_size)
    return fail(KVQ_ERR_SHAPE, "%s: the K and V pools differ in heads/dim/page_size", fn);
  const int D = p0.head_dim, H = p0.num_heads;
  if (D != 64 && D != 128 && D != 256)
    return fail(KVQ_ERR_SHAPE, "%s: head_dim %d is none of 64, 128, 256", fn, D);
  if (p0.page_size % kTile != 0)
    return fail(KVQ_ERR_SHAPE, "%s: page_size %d is not a multiple of %d", fn, p0.page_size, kTile);
  if (num_q_heads < 1 || num_q_heads % H != 0 || num_q_heads / H > 64)
    return fail(KVQ_ERR_SHAPE, "%s: %d query heads over %d KV heads", fn, num_q_heads, H);
  if (beams < 1 || beams > KVQ_MAX_BEAMS)
    return fail(KVQ_ERR_SHAPE, "%s: beams %d not in [1, %d]", fn, beams, KVQ_MAX_BEAMS);
  if (nseq < 0 || nseq > KVQ_MAX_SEQS || nseq % beams != 0)
    return fail(KVQ_ERR_RANGE, "%s: nseq %d must be a multiple of beams, at most %d", fn, nseq,
                KVQ_MAX_SEQS);
  // The longest prefix and the longest own part may be of different groups; that a row of the table holds their
  // sum is asked for all the same, as a check of the bounds, unless max_own is all that it holds.
  const int max_len =
      static_cast<int>(std::min<int64_t>(static_cast<int64_t>(max_pages) * p0.page_size, kMostTokens));
  if (max_pages < 1 || max_shared < 0 || max_own < 0 || max_shared > max_len || max_own > max_len ||
      (static_cast<int64_t>(max_shared) + max_own > max_len && max_own != max_len))
    return fail(KVQ_ERR_RANGE, "%s: max_shared %d, max_own %d where a row of the table holds %d tokens", fn,
                max_shared, max_own, max_len);
  if (!shared_lens && max_shared != 0)
    return fail(KVQ_ERR_NULL, "%s: max_shared without shared_lens", fn);
  if (!(softmax_scale > 0.f && softmax_scale <= 2.3e38f))
    return fail(KVQ_ERR_RANGE, "%s: softmax_scale %g", fn, static_cast<double>(softmax_scale));
  if (nseq == 0) return ok();
  if (!q || !page_table || !seq_lens || !out || !workspace)
    return fail(KVQ_ERR_NULL, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(KVQ_ERR_ALIGN, "%s: q, out and workspace must be 16-byte aligned", fn);
  const size_t need = kvq_beam_attn_workspace(n_layers, nseq, beams, H, num_q_heads, D, max_shared, max_own);
  if (workspace_bytes < need)
    return fail(KVQ_ERR_WORKSPACE, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  const Plan p = plan(n_layers, nseq, beams, H, num_q_heads, D, max_shared, max_own);
  if (static_cast<int64_t>(n_layers) * H > INT32_MAX ||
      static_cast<int64_t>(n_layers) * nseq * num_q_heads > INT32_MAX)
    return fail(KVQ_ERR_RANGE, "%s: %d layers of %d sequences and %d heads", fn, n_layers, nseq, num_q_heads);
  BeamArgs a;
  for (int i = 0; i < KVQ_MAX_TENSORS; ++i)
    a.L[i] = i < n_layers ? LayerPools{k_pools[i].codes, k_pools[i].scales, v_pools[i].codes,
                                       v_pools[i].scales,
                                       std::min(k_pools[i].num_pages, v_pools[i].num_pages)}
                          : LayerPools{};
  a.q = q; a.out = out;
  a.head = static_cast<int64_t*>(workspace);
  a.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + p.head_bytes());
  a.pt = page_table; a.lens = seq_lens; a.shared = shared_lens; a.err = dev_err;
  a.nseq = nseq; a.beams = beams; a.groups = nseq / beams;
  a.H = H; a.G = num_q_heads / H; a.Hq = num_q_heads; a.ps = p0.page_size;
  a.max_pages = max_pages; a.n_layers = n_layers;
  a.line[0] = p.line[0]; a.line[1] = p.line[1];
  a.max_shared = max_shared; a.max_own = max_own; a.max_len = max_len;
  a.magic = 0x64006400u;
  a.scale = softmax_scale * 1.4426950408889634f;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == KVQ_BF16 ? run_bf16(a, D, p.nt, p.granules, cs)
                                          : run_f16(a, D, p.nt, p.granules, cs);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return ok();
}
