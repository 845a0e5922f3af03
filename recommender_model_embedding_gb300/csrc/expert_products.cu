// The experts' products from their parts: which operands the tensor cores can read where they lie, which
// are copied first, and the launches in order.
#include <algorithm>

#include "expert_few.cuh"

namespace emb {

namespace {

// Pieces of the workspace, one after the other on 128-byte boundaries (from no base: their sizes).
struct Room {
  char* base;
  int64_t used = 0;
  template <typename T>
  T* take(int64_t count) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (count * (int64_t)sizeof(T) + 127) / 128 * 128;
    return base ? p : nullptr;
  }
};

struct Source {
  const void* p;
  int64_t inner, rows, ld, half_step, expert_step;
  int halves = 1, experts = 1;
  const int32_t* last = nullptr;
};

// Room for an operand of the tensor cores: row steps on 16 bytes, three planes for fp32.
MmOperand packed(Room& room, int64_t inner, int64_t rows, int halves, int experts, int planes) {
  MmOperand o;
  o.inner = inner, o.rows = rows, o.halves = halves, o.experts = experts, o.planes = planes;
  o.ld = (inner + 7) / 8 * 8;
  o.half_step = rows * o.ld, o.expert_step = halves * o.half_step, o.plane_step = experts * o.expert_step;
  o.p = room.take<__nv_bfloat16>(o.planes * o.plane_step);
  return o;
}

// The copies that a call begins with.
struct Packs {
  PackArgs list[kMaxPacks];
  int count = 0;
};

// A matrix as the tensor cores take it: in place, or as a copy.  One matrix for all experts is one matrix.
MmOperand operand(Source m, bool f32, Room& room, Packs& packs) {
  MmOperand o;
  if (m.expert_step == 0) m.experts = 1;
  if (!f32 && reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (m.rows <= 1 || (m.ld % 8 == 0 && m.ld >= m.inner)) &&
      (m.halves == 1 || (m.half_step % 8 == 0 && m.half_step > 0)) &&
      (m.experts == 1 || (m.expert_step % 8 == 0 && m.expert_step < (int64_t)1 << 38))) {
    o.p = static_cast<const __nv_bfloat16*>(m.p);
    o.inner = m.inner, o.rows = m.rows, o.ld = m.ld, o.half_step = m.half_step, o.expert_step = m.expert_step;
    o.halves = m.halves, o.experts = m.experts;
    return o;
  }
  o = packed(room, m.inner, m.rows, m.halves, m.experts, f32 ? 3 : 1);
  PackArgs& a = packs.list[packs.count++];
  a.src = m.p, a.ld = m.ld, a.half_step = m.half_step, a.expert_step = m.expert_step;
  a.f32 = f32, a.last = m.last, a.to = o;
  return o;
}

// What the tiles of an M x N weight gradient take, in fifths of one of 256 x 256 (one of 128 columns: three).
int64_t tile_cost(int64_t M, int64_t N) {
  return (M + 255) / 256 * std::min(5 * ((N + 255) / 256), 3 * ((N + 127) / 128));
}

// Tiles of a weight gradient with M x N outputs: narrower ones, or rows cut into parts, where the
// experts' tiles alone leave pairs of SMs without work.  A part's rows are such that one dense layer's tiles
// fill the pairs once, and several experts' (which have unlike numbers of rows) about twice.
void cut_wgrad(MmArgs& a, int64_t rows) {
  const int64_t pairs = mm_pairs();
  const auto tiles = [&](int n) { return (int64_t)((a.M + 255) / 256) * ((a.N + n - 1) / n); };
  // (a tile of 128 columns takes about 0.6 of the time of one of 256)
  a.tile_n = 5 * tiles(256) > 3 * tiles(128) ? 128 : 256, a.split = 0;
  const int64_t each = tiles(a.tile_n);
  if (a.E * each >= pairs) return;
  // A tile takes 0.15 to 0.27 us for 64 rows and product of planes, parts a launch and their sum, some 6 us: where
  // rows are so few that parts would not save that, tiles of half the columns (all SMs busy, those are bound by their
  // loads and no faster: 16411 x 1000 x 479 in bf16 30 us with them and 4 parts).
  const int terms = a.f32 ? 6 : std::max(a.a.planes, a.b.planes);
  if (rows * terms < (int64_t)a.E * 64 * 80) {
    a.tile_n = 128;
    return;
  }
  const int64_t parts = a.E == 1 ? pairs / each : 2 * pairs / each;
  const int64_t cut = std::max<int64_t>(256, (rows / parts + 63) / 64 * 64);
  if (cut * a.E < rows) a.split = (int)cut;
}

// Whether the kernel for few rows is the faster, by what both take (microseconds, weights in MB; measured over 1 to
// 128 experts, widths 128 to 2048, 1 to 256 rows an expert, both layouts): that kernel reads the weights once for
// every 32 rows of an expert, at a rate that falls with the rows it multiplies them by (64 experts of 1024 x
// 512 in bf16: 15 us with 8 rows, 22 with 16, 32 with 32); the tiles' kernel takes longer to get going and
// some 3 us for a tile, and reads them once for 256 rows (16 us for all three), for fp32 after copying them as
// bf16 planes.  The host knows the rows' number and not whose they are, so all of it goes by the average: where most
// rows are one expert's, this kernel reads that expert's weights (from L2) again for every 8, 16 or 32 of them.
bool few(int64_t rows, int experts, int64_t outs, int64_t in, bool f32) {
  const int64_t each = (rows + experts - 1) / experts, passes = (each + 31) / 32;
  if (each > 128 || few_tiles(rows, experts, 8) > 65535) return false;
  const double mb = 1e-6 * (double)(std::min<int64_t>(experts, rows) * outs * in) * (f32 ? 4 : 2);
  const double rate = f32 ? (each <= 8 ? 0.75 : each <= 16 ? 1.0 : 1.4) : (each <= 8 ? 0.19 : each <= 16 ? 0.30 : 0.43);
  const double all = 1e-6 * (double)(experts * outs * in) * (f32 ? 4 : 2);  // (copies go over all experts' weights)
  const double tiles = (double)((outs + 255) / 256 * std::min<int64_t>(experts, rows)) / (double)mm_pairs();
  return 2.5 + (double)passes * mb * rate < (f32 ? 10.5 + 0.9 * all : 6.0 + std::max(0.15 * mb, 3.0 * (tiles - 1)));
}

cudaError_t product(const emb_product& p, ProductKind kind, Room& room, bool launch, cudaStream_t s) {
  const bool f32 = p.dtype == EMB_F32, gated = kind == kGated || kind == kGatedBackward;
  const bool back = kind == kLinearBackward || kind == kGatedBackward;
  const int64_t S = p.rows, in = p.in, f = p.out, O = gated ? 2 * f : f;
  const int32_t* last = p.d_offsets ? p.d_offsets + p.experts : nullptr;
  cudaError_t e = cudaSuccess;
  Packs packs;
  MmArgs a;
  a.offsets = p.d_offsets, a.E = p.experts, a.S = (int)S, a.f32 = f32;
  const Source x{p.d_x, in, S, p.x_ld, 0, 0, 1, 1, last};
  if (!back) {
    if (S == 0) return cudaSuccess;
    if (few(S, p.experts, O, in, f32)) {
      FewArgs w;
      w.offsets = p.d_offsets, w.E = p.experts, w.S = (int)S, w.in = (int)in, w.out = (int)f, w.act = gated ? p.act : -1;
      w.f32 = f32, w.turned = p.w_turned != 0;
      w.x = p.d_x, w.x_ld = p.x_ld, w.w = p.d_w, w.w_ld = p.w_ld, w.w_step = p.w_step;
      w.half = gated ? (p.w_turned ? f : f * p.w_ld) : 0;
      w.y = p.d_out, w.y_ld = p.out_ld;
      if (gated) w.gu = p.d_gu, w.gu_ld = p.gu_ld;
      return launch ? launch_expert_few(w, s) : cudaSuccess;
    }
    Source w{p.d_w, p.w_turned ? f : in, p.w_turned ? in : f, p.w_ld, p.w_turned ? f : f * p.w_ld, p.w_step, gated ? 2 : 1, p.experts};
    a.a = operand(x, f32, room, packs), a.b = operand(w, f32, room, packs);
    if (!launch) return cudaSuccess;
    if ((e = launch_expert_packs(packs.list, packs.count, s)) != cudaSuccess) return e;
    a.b_mn = p.w_turned != 0;
    a.N = (int)f, a.K = (int)in, a.act = gated ? p.act : -1;
    a.out = p.d_out, a.out_ld = p.out_ld, a.out_bf16 = !f32;
    if (gated) a.gu = p.d_gu, a.gu_ld = p.gu_ld;
    return launch_expert_mm_rows(a, s);
  }
  // [dg, du], or dout; of bf16 rows an fp32 dw takes all planes of dg and du, dx and a bf16 dw two
  MmOperand d, xo, wo;
  const bool dx = p.d_dx && S > 0;
  if (S > 0) {
    if (gated) d = packed(room, O, S, 1, 1, f32 || (p.d_dw && p.dw_dtype == EMB_F32) ? 3 : 2);
    else d = operand({p.d_dout, f, S, p.dout_ld, 0, 0, 1, 1, last}, f32, room, packs);
    if (dx) wo = operand({p.d_w, p.w_turned ? O : in, p.w_turned ? in : O, p.w_ld, 0, p.w_step, 1, p.experts}, f32, room, packs);
    if (p.d_dw) xo = operand(x, f32, room, packs);
    if (launch && packs.count && (e = launch_expert_packs(packs.list, packs.count, s)) != cudaSuccess) return e;
    if (launch && gated && (e = launch_expert_gated_bwd(p, d, packs.count > 0, s)) != cudaSuccess) return e;
  }
  if (dx) {
    a.a = d, a.b = wo;
    if (!f32) a.a.planes = gated ? 2 : 1;
    a.b_mn = p.w_turned == 0;
    a.N = (int)in, a.K = (int)O;
    a.out = p.d_dx, a.out_ld = p.dx_ld, a.out_bf16 = !f32;
    if (launch && (e = launch_expert_mm_rows(a, s)) != cudaSuccess) return e;
  }
  if (p.d_dw) {
    // dw as it lies, or the other way round where that takes less of tiles of 256 x 256 (or 0.6 for 128)
    const bool first = p.dw_turned ? tile_cost(O, in) < tile_cost(in, O) : tile_cost(O, in) <= tile_cost(in, O);  // O x in
    a.a = first ? d : xo, a.b = first ? xo : d;
    a.M = (int)(first ? O : in), a.N = (int)(first ? in : O), a.K = 0;
    a.turned = first == (p.dw_turned != 0);
    a.out = p.d_dw, a.out_ld = p.dw_ld, a.out_step = p.dw_step, a.out_bf16 = p.dw_dtype == EMB_BF16;
    cut_wgrad(a, S);
    a.beside = dx;
    if (a.split) a.parts = room.take<float>((S / a.split + std::min<int64_t>(p.experts, S)) * a.M * a.N);
    if (launch) return launch_expert_mm_wgrad(a, s);
  }
  return e;
}

}  // namespace

int64_t expert_product_workspace(const emb_product& p, ProductKind kind) {
  Room room{nullptr};
  product(p, kind, room, false, nullptr);
  return room.used;
}

cudaError_t launch_expert_product(const emb_product& p, ProductKind kind, void* ws, cudaStream_t s) {
  Room room{static_cast<char*>(ws)};
  return product(p, kind, room, true, s);
}

}  // namespace emb
