// The global norm of a list of gradients, and clipping by it.
//
// norm = sqrt(sum over all tensors of g^2); out = g min(1, max_norm / (norm +
// 1e-6)). The factor depends on every element, so the gradients are read
// twice and written once: bound by memory. Squares are summed in 64 bits (two
// more instructions an element, far under the memory's rate), so no square
// over- or underflows, and in a fixed order, so results repeat bit for bit.
//
// The tensors are cut into chunks. The list reaches the first kernel by value,
// kTensors a launch (a launch's arguments end at 4 KB): it sums the squares of
// its chunks and leaves in the workspace one partial sum a workgroup and one
// record a chunk (address, place in the output, length). The second kernel
// takes all records of all launches: every workgroup forms the norm from the
// partial sums in the same order, then scales its chunks. 448 tensors of 40 M
// float32 in all: 40 us for the norm (two launches, 4.0 TB/s), 67 us more for the
// scaling into a second buffer (320 MB, 4.8 TB/s, a large copy's rate). Replayed
// on one set of tensors, whose 160 MB partly stay in the 256 MB cache: 35 us the
// norm, 86 us with the scaling, 84 us in place.
#include "elem.h"

namespace qlora {
namespace {

constexpr int kTensors = 240;
constexpr int kThreads = 256;
constexpr int kRun = 8;                         // elements of a thread at a time
constexpr int kTurns = 4;                       // runs of a thread in a chunk, at most
constexpr int kSmallChunk = kThreads * kRun;    // 2048
constexpr int kChunk = kSmallChunk * kTurns;    // 8192
constexpr int kSumBlocks = 1024;                // workgroups of a first launch, at most
constexpr int kScaleBlocks = 1024;              // of the second

// A launch's tensors. Tensor i's chunks are first[i] .. first[i + 1] - 1,
// counted from the launch's first; pad[i] elements are missing from the chunks
// in front of it, so its elements in front in the list, and its length, follow.
struct Slice {
  const void* at[kTensors];
  int32_t first[kTensors + 1];
  int32_t pad[kTensors + 1];
};
static_assert(sizeof(Slice) <= 3900, "kernel arguments end at 4 KB");

struct Record {
  const void* at;
  int64_t off;
  int64_t len;
};

// Sum over the workgroup in a fixed order, in every thread.
__device__ __forceinline__ double reduce_sum(double v) {
  __shared__ double sums[kThreads / 64];
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kThreads / 64; ++i) v += sums[i];
  return v;
}

// A thread's runs of a chunk: run i starts at element kRun (thread + i
// kThreads); what lies behind the chunk's end is zero. A whole chunk is loaded
// without a branch, all runs in flight at once.
template <int kType>
__device__ __forceinline__ void load_chunk(const typename Elem<kType>::T* p, int64_t len, float (*v)[kRun]) {
  if (len == kChunk) {
    Words8<kType> w[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) w[i] = load8<kType>(p + kRun * (threadIdx.x + i * kThreads));
#pragma unroll
    for (int i = 0; i < kTurns; ++i) values8<kType>(w[i], v[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int64_t j = kRun * (threadIdx.x + i * kThreads);
    if (j + kRun <= len) {
      values8<kType>(load8<kType>(p + j), v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[i][e] = j + e < len ? Elem<kType>::get(p[j + e]) : 0.0f;
    }
  }
}

template <int kType>
__global__ __launch_bounds__(kThreads) void square_sum_kernel(Slice l, int tensors, int chunk, int64_t off0,
                                                              double* partial, Record* records) {
  typedef typename Elem<kType>::T T;
  const int lane = threadIdx.x & 63;
  double sum = 0.0;
  const int chunks = l.first[tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    // the last tensor that starts at or in front of chunk c: the starts ascend
    int t = -1;
#pragma unroll
    for (int j = 0; j < kTensors; j += 64)
      t += __popcll(__ballot(j + lane < tensors && l.first[j + lane < kTensors ? j + lane : 0] <= c));
    t = __builtin_amdgcn_readfirstlane(t);
    const int64_t begin = static_cast<int64_t>(c - l.first[t]) * chunk;
    const int len = c + 1 < l.first[t + 1] ? chunk : chunk - (l.pad[t + 1] - l.pad[t]);
    const T* p = static_cast<const T*>(l.at[t]) + begin;
    if (records != nullptr && threadIdx.x == 0)
      records[c] = Record{p, off0 + static_cast<int64_t>(c) * chunk - l.pad[t], len};
    float v[kTurns][kRun];
    load_chunk<kType>(p, len, v);
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
      for (int e = 0; e < kRun; ++e) sum += static_cast<double>(v[i][e]) * static_cast<double>(v[i][e]);
  }
  sum = reduce_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// clip = false: only the norm (one workgroup). out null: in place. The first
// chunk is on its way while the partial sums are added.
template <int kType>
__global__ __launch_bounds__(kThreads) void scale_kernel(const double* partial, int partials, const Record* records,
                                                         int chunks, bool clip, float max_norm, void* out,
                                                         float* norm_out) {
  typedef typename Elem<kType>::T T;
  int c = blockIdx.x;
  Record r{};
  float v[kTurns][kRun];
  if (clip && c < chunks) {
    r = records[c];
    load_chunk<kType>(static_cast<const T*>(r.at), r.len, v);
  }
  double sum = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  const double norm = sqrt(reduce_sum(sum));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  if (!clip) return;
  float f = 1.0f;
  const double ratio = static_cast<double>(max_norm) / (norm + 1e-6);
  if (!(ratio >= 1.0) && !__builtin_isinf(max_norm)) f = static_cast<float>(ratio);  // a NaN norm: NaN
  if (out == nullptr && f == 1.0f) return;
  while (c < chunks) {
    T* o = out == nullptr ? static_cast<T*>(const_cast<void*>(r.at)) : static_cast<T*>(out) + r.off;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int64_t j = kRun * (threadIdx.x + i * kThreads);
#pragma unroll
      for (int e = 0; e < kRun; ++e) v[i][e] *= f;
      if (j + kRun <= r.len) {
        put8<kType>(o + j, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
          if (j + e < r.len) o[j + e] = Elem<kType>::put(v[i][e]);
      }
    }
    c += gridDim.x;
    if (c >= chunks) return;
    r = records[c];
    load_chunk<kType>(static_cast<const T*>(r.at), r.len, v);
  }
}

// Chunk length and what follows from it.
struct Plan {
  int chunk;
  int chunks;    // of all tensors
  int partials;  // workgroups of all first launches
};

int64_t chunks_of(int64_t numel, int chunk) { return (numel + chunk - 1) / chunk; }

Plan plan_for(const int64_t* numel, int count) {
  int64_t total = 0;
  for (int i = 0; i < count; ++i) total += numel[i];
  Plan p{};
  p.chunk = total < kChunk * 512 ? kSmallChunk : kChunk;  // short lists: chunks for every CU
  int64_t chunks = 0, in_slice = 0;
  int tensors = 0;
  for (int i = 0; i < count; ++i) {
    if (numel[i] == 0) continue;
    const int64_t c = chunks_of(numel[i], p.chunk);
    chunks += c;
    in_slice += c;
    if (++tensors == kTensors) {
      p.partials += static_cast<int>(in_slice < kSumBlocks ? in_slice : kSumBlocks);
      tensors = 0;
      in_slice = 0;
    }
  }
  if (tensors > 0) p.partials += static_cast<int>(in_slice < kSumBlocks ? in_slice : kSumBlocks);
  p.chunks = static_cast<int>(chunks);
  return p;
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

template <int kType>
hipError_t launch_t(const void* const* grads, const int64_t* numel, int count, bool clip, float max_norm, void* out,
                    float* norm, void* ws, hipStream_t s) {
  const Plan p = plan_for(numel, count);
  double* partial = static_cast<double*>(ws);
  Record* records = reinterpret_cast<Record*>(static_cast<char*>(ws) + up256(p.partials * 8));
  Slice l{};
  int tensors = 0, chunks = 0, partials = 0;
  int64_t off = 0, off0 = 0;  // elements in front of the next tensor, of the launch
  for (int i = 0; i <= count; ++i) {
    if (i < count && numel[i] > 0) {
      const int64_t n = chunks_of(numel[i], p.chunk);
      l.at[tensors] = grads[i];
      l.first[tensors + 1] = l.first[tensors] + static_cast<int32_t>(n);
      l.pad[tensors + 1] = l.pad[tensors] + static_cast<int32_t>(n * p.chunk - numel[i]);
      off += numel[i];
      ++tensors;
    }
    if (tensors == kTensors || (i == count && tensors > 0)) {
      const int mine = l.first[tensors], blocks = mine < kSumBlocks ? mine : kSumBlocks;
      hipLaunchKernelGGL((square_sum_kernel<kType>), dim3(blocks), dim3(kThreads), 0, s, l, tensors, p.chunk, off0,
                         partial + partials, clip ? records + chunks : nullptr);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      partials += blocks;
      chunks += mine;
      off0 = off;
      tensors = 0;
    }
  }
  int blocks = clip ? (p.chunks < kScaleBlocks ? p.chunks : kScaleBlocks) : 1;
  if (blocks < 1) blocks = 1;
  hipLaunchKernelGGL((scale_kernel<kType>), dim3(blocks), dim3(kThreads), 0, s, partial, partials, records, p.chunks,
                     clip, max_norm, out, norm);
  return hipGetLastError();
}

}  // namespace

size_t grad_ws_bytes(const int64_t* numel, int count) {
  const Plan p = plan_for(numel, count);
  return static_cast<size_t>(up256(p.partials * 8) + up256(static_cast<int64_t>(p.chunks) * sizeof(Record)));
}

hipError_t launch_grad_clip(const void* const* grads, const int64_t* numel, int count, int dtype, bool clip,
                            float max_norm, void* out, float* norm, void* ws, hipStream_t s) {
  auto fn = dtype == QLORA_F32 ? launch_t<QLORA_F32> : dtype == QLORA_F16 ? launch_t<QLORA_F16> : launch_t<QLORA_BF16>;
  return fn(grads, numel, count, clip, max_norm, out, norm, ws, s);
}

}  // namespace qlora
