// The C ABI of the bf16 paged cache and of the drafts' check (declared in include/dsa.h): argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <limits>
#include <numeric>

#include "../../include/dsa.h"
#include "api_checks.h"
#include "launch.h"
#include "paged.cuh"

namespace dsa {
namespace {

dsa_status check_table(PageTable* c, const int32_t* table, int R, int M, int P, int page_rows) {
  if (P < 0 || R < 0 || M < 0) return DSA_ERR_INVALID_ARG;
  if (!paged_rows(page_rows)) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(M) * page_rows > INT_MAX) return DSA_ERR_UNSUPPORTED;  // a row's position is an int
  if (static_cast<int64_t>(R) * M > 0 && (!table || !aligned(table, 4))) return DSA_ERR_INVALID_ARG;
  *c = PageTable{table, P, R, M, log2_of(page_rows)};
  return DSA_OK;
}

// The two ways in which the (token, head) rows of a call may be cut into units of at most N rows.  Whole tokens, m a unit (or a
// token's heads in equal units of their own): no token has its rows walked over twice, and up to half of the columns are idle.  Or
// N rows wherever they begin: no column is idle, and a token in two units has its rows walked over by both.  A run of k tokens of
// a sequence is walked over by (k + m - 1) / m units (k of each of its groups) or by (k H + N - gcd(H, N)) / N, on the average over its
// place, so the better one depends on how many tokens share a sequence: the kernel counts them (places without a token, and the
// table's height, say nothing) and takes the cut with fewer walks.  Measured, whole and anywhere: 64 sequences of 4096 rows, a token each,
// 150 heads of 256 75 and 89 us, 100 heads of 512 112 and 118, 20 heads of 128 40.9 and 42.9; 200 tokens over 8192 rows, 150
// heads of 256 272 and 182, 65 heads of 128 86 and 59, 40 heads of 512 207 and 144.
struct Cuts {
  PagedCut whole, any;
  float per_token, per_run;
};
PagedCut cut_of(int64_t rows, int groups, int T, int H) {
  const int64_t units = groups > 1 ? static_cast<int64_t>(T) * groups : (static_cast<int64_t>(T) * H + rows - 1) / rows;
  return {static_cast<int>(rows), groups, static_cast<int>(units)};
}
Cuts cuts_of(int T, int H, int D) {
  const int N = paged_attn_cols(D);
  const int tokens = H <= N ? std::min(kPagedMaxTokens, N / H) : 0;  // m
  const int groups = H <= N ? 1 : H / N + (H % N != 0 ? 1 : 0);
  Cuts c;
  c.whole = H <= N ? cut_of(tokens * H, 1, T, H) : cut_of(H / groups + (H % groups != 0 ? 1 : 0), groups, T, H);
  // (no choice: a token alone, heads that fill N, more tokens than a unit of any N rows may hold: n rows lie in n / H + 2 of them)
  const bool same = T == 1 || (H <= N && N % H == 0) || N / H + 2 > kPagedMaxTokens;
  c.any = same ? c.whole : cut_of(N, 1, T, H);
  const float n = static_cast<float>(N), h = static_cast<float>(H), m = static_cast<float>(tokens);
  c.per_token = h / n - (H <= N ? 1.f / m : static_cast<float>(groups));
  c.per_run = static_cast<float>(N - std::gcd(H, N)) / n - (H <= N ? (m - 1.f) / m : 0.f);
  return c;
}

struct Workspace {
  size_t partial, stats, bytes;  // offsets of the parts behind the shared units' entries
};
Workspace workspace_of(int D, int ctas) {
  const size_t n = paged_attn_cols(D);
  Workspace w;
  w.partial = static_cast<size_t>(ctas) * sizeof(int4);
  w.stats = w.partial + 2 * static_cast<size_t>(ctas) * n * D * sizeof(float);
  w.bytes = w.stats + 2 * static_cast<size_t>(ctas) * 2 * n * sizeof(float);
  return w;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_step_maps(const int32_t* held, const int32_t* added, int R, int T, int32_t* seq, int32_t* pos, int32_t* ks,
                         int32_t* ke, void* stream) {
  if (R < 0 || T < 0) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (R > 0 && (!held || !aligned(held, 4) || !added || !aligned(added, 4))) return DSA_ERR_INVALID_ARG;
  if (!seq || !aligned(seq, 4) || !pos || !aligned(pos, 4) || !ks || !aligned(ks, 4) || !ke || !aligned(ke, 4))
    return DSA_ERR_INVALID_ARG;
  int32_t* const maps[4] = {seq, pos, ks, ke};
  for (int i = 0; i < 4; ++i) {
    if (overlap(maps[i], T, held, R) || overlap(maps[i], T, added, R)) return DSA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(maps[i], T, maps[j], T)) return DSA_ERR_INVALID_ARG;
  }
  return done(launch_step_maps(StepMapArgs{held, added, R, T, seq, pos, ks, ke}, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_page_slots(const int32_t* table, int R, int M, int P, int page_rows, const int32_t* seq, const int32_t* start,
                          const int32_t* idx, int T, int K, int32_t* slots, void* stream) {
  PageTable c;
  const dsa_status st = check_table(&c, table, R, M, P, page_rows);
  if (st != DSA_OK) return st;
  if (T < 0 || K < 0) return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(P) * page_rows > INT_MAX) return DSA_ERR_UNSUPPORTED;  // a row of the pages is an int
  if (T == 0 || K == 0) return DSA_OK;
  if (!seq || !aligned(seq, 4) || !idx || !aligned(idx, 4) || !slots || !aligned(slots, 4) || (start && !aligned(start, 4)))
    return DSA_ERR_INVALID_ARG;
  const int64_t entries = static_cast<int64_t>(T) * K;
  if ((slots != idx && overlap(slots, entries, idx, entries)) || overlap(slots, entries, seq, T) ||
      (start && overlap(slots, entries, start, T)) || overlap(slots, entries, table, static_cast<int64_t>(R) * M))
    return DSA_ERR_INVALID_ARG;
  return done(launch_page_slots(c, seq, start, idx, T, K, slots, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_store_kv(const uint16_t* kv, int64_t stride, const int32_t* seq, const int32_t* pos, int N, int D, uint16_t* pages,
                        int P, int page_rows, const int32_t* table, int R, int M, const int32_t* lacking, void* stream) {
  PageTable c;
  const dsa_status st = check_table(&c, table, R, M, P, page_rows);
  if (st != DSA_OK) return st;
  if (!paged_d(D)) return DSA_ERR_UNSUPPORTED;
  if (P > 0 && (!pages || !aligned(pages, 16))) return DSA_ERR_INVALID_ARG;
  if (N < 0 || (N > 1 && (stride < D || stride > (INT64_MAX >> 2) / N)) || stride % 8 != 0) return DSA_ERR_INVALID_ARG;
  if (N == 0) return DSA_OK;
  if (!kv || !aligned(kv, 16) || !seq || !aligned(seq, 4) || !pos || !aligned(pos, 4) || (lacking && !aligned(lacking, 4)))
    return DSA_ERR_INVALID_ARG;
  const int64_t held = static_cast<int64_t>(P) * page_rows * D;
  if (overlap(pages, held, kv, (N - 1) * stride + D) || overlap(pages, held, seq, N) || overlap(pages, held, pos, N) ||
      overlap(pages, held, table, static_cast<int64_t>(R) * M) || overlap(pages, held, lacking, lacking ? 1 : 0))
    return DSA_ERR_INVALID_ARG;
  return done(launch_store_kv(D, kv, stride, N, seq, pos, lacking, pages, c, static_cast<cudaStream_t>(stream)));
}

size_t dsa_paged_attn_workspace_size(int T, int H, int D) {
  DeviceFacts dev;
  if (T <= 0 || H < 1 || !paged_d(D) || !device_facts(&dev)) return 0;
  return workspace_of(D, dev.sms).bytes;
}

dsa_status dsa_paged_attn(const uint16_t* q, const uint16_t* pages, int P, int page_rows, const int32_t* table, int R, int M,
                          const int32_t* seq, const int32_t* pos, const float* attn_sink, int T, int H, int D, int window,
                          int first, float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
  PageTable c;
  const dsa_status st = check_table(&c, table, R, M, P, page_rows);
  if (st != DSA_OK) return st;
  if (!paged_d(D)) return DSA_ERR_UNSUPPORTED;
  if (T < 0 || H < 1 || window < 0 || first < 0) return DSA_ERR_INVALID_ARG;
  if (P > 0 && (!pages || !aligned(pages, 16))) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!q || !aligned(q, 16) || !out || !aligned(out, 16) || !seq || !aligned(seq, 4) || !pos || !aligned(pos, 4))
    return DSA_ERR_INVALID_ARG;
  if ((attn_sink && !aligned(attn_sink, 4)) || (lse && !aligned(lse, 4))) return DSA_ERR_INVALID_ARG;
  // rows of q and of the pages are coordinates of the copies, which are ints (and there are no more units than rows of q)
  if (static_cast<int64_t>(T) * H > INT_MAX / 2 || static_cast<int64_t>(P) * page_rows > INT_MAX)
    return DSA_ERR_UNSUPPORTED;
  const int64_t values = static_cast<int64_t>(T) * H * D, held = static_cast<int64_t>(P) * page_rows * D;
  const int64_t logs = lse ? static_cast<int64_t>(T) * H : 0, entries = static_cast<int64_t>(R) * M, sinks = attn_sink ? H : 0;
  if ((out != q && overlap(out, values, q, values)) || overlap(out, values, lse, logs) || overlap(lse, logs, q, values))
    return DSA_ERR_INVALID_ARG;
  const auto taken = [&](const auto* o, int64_t n) {
    return overlap(o, n, pages, held) || overlap(o, n, table, entries) || overlap(o, n, seq, T) || overlap(o, n, pos, T) ||
           overlap(o, n, attn_sink, sinks);
  };
  if (taken(out, values) || taken(lse, logs)) return DSA_ERR_INVALID_ARG;
  DeviceFacts dev;
  if (!device_facts(&dev)) return DSA_ERR_CUDA;
  if (paged_attn_smem(D) > dev.max_smem) return DSA_ERR_UNSUPPORTED;
  const Workspace w = workspace_of(D, dev.sms);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < w.bytes) return DSA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t bytes = static_cast<int64_t>(w.bytes);
  if (taken(ws, bytes) || overlap(ws, bytes, q, values) || overlap(ws, bytes, out, values) || overlap(ws, bytes, lse, logs))
    return DSA_ERR_INVALID_ARG;
  const int box = std::min(page_rows, paged_attn_block(D));
  CUtensorMap kvmap, qmap;
  // (without pages the map is over q, of which no row of a page is read)
  if (!make_bf16_map(&kvmap, P > 0 ? pages : q, P > 0 ? static_cast<int64_t>(P) * page_rows : 1, D, box) ||
      !make_bf16_map(&qmap, q, static_cast<int64_t>(T) * H, D, paged_attn_cols(D)))
    return DSA_ERR_CUDA;
  const Cuts cuts = cuts_of(T, H, D);
  // (at D <= 256 a scale of 0 is the least number, 2^-149, so that what is masked stays minus infinity: the largest score becomes 2^-21)
  float to_log2 = scale * 1.4426950408889634f;
  if (to_log2 == 0.f && D <= 256) to_log2 = std::numeric_limits<float>::denorm_min();
  PagedAttnParams p{c, seq, pos, attn_sink, out, lse, reinterpret_cast<float*>(ws + w.partial),
                    reinterpret_cast<float*>(ws + w.stats), reinterpret_cast<int4*>(ws), T, H, cuts.whole, cuts.any,
                    cuts.any.rows != cuts.whole.rows && T > R ? 1 : 0, cuts.per_token, cuts.per_run,
                    window == 0 ? INT_MAX : window, first, box, {to_log2, to_log2}, 0u, 0};
  p.set_heads(H);
  return done(launch_paged_attn(D, dev.sms, kvmap, qmap, p, dev.err, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_verify_drafts(const float* target, const float* draft, const int32_t* tokens, const int32_t* count,
                             const float* u, int R, int G, int V, int32_t* accepted, int32_t* token, void* stream) {
  if (R < 0 || G < 0 || V < 1) return DSA_ERR_INVALID_ARG;
  if (R > INT_MAX / 8 || G == INT_MAX) return DSA_ERR_UNSUPPORTED;  // CTAs of a launch; G + 1
  if (R == 0) return DSA_OK;
  if (!target || !aligned(target, 4) || !count || !aligned(count, 4) || !u || !aligned(u, 4) || !accepted || !aligned(accepted, 4) ||
      !token || !aligned(token, 4))
    return DSA_ERR_INVALID_ARG;
  if (G > 0 && (!draft || !aligned(draft, 4) || !tokens || !aligned(tokens, 4))) return DSA_ERR_INVALID_ARG;
  const int64_t drafts = static_cast<int64_t>(R) * G;
  if (drafts + R > (INT64_MAX >> 3) / V) return DSA_ERR_UNSUPPORTED;  // the probabilities' bytes
  for (int32_t* o : {accepted, token})
    if (overlap(o, R, count, R) || overlap(o, R, tokens, drafts) || overlap(o, R, u, drafts + R) ||
        overlap(o, R, target, (drafts + R) * V) || overlap(o, R, draft, drafts * V))
      return DSA_ERR_INVALID_ARG;
  if (overlap(accepted, R, token, R)) return DSA_ERR_INVALID_ARG;
  DeviceFacts dev;
  if (!device_facts(&dev)) return DSA_ERR_CUDA;
  return done(launch_verify_drafts(VerifyArgs{target, draft, tokens, count, u, R, G, V, accepted, token}, dev.sms,
                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
