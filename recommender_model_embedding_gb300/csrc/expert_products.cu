// The experts' products from their parts: which operands the tensor cores can read where they lie, which
// are copied first, and the launches in order.
#include <algorithm>

#include "expert_mm.cuh"

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
MmOperand packed(Room& room, int64_t inner, int64_t rows, int halves, int experts, bool f32) {
  MmOperand o;
  o.inner = inner, o.rows = rows, o.halves = halves, o.experts = experts, o.planes = f32 ? 3 : 1;
  o.ld = (inner + 7) / 8 * 8;
  o.half_step = rows * o.ld, o.expert_step = halves * o.half_step, o.plane_step = experts * o.expert_step;
  o.p = room.take<__nv_bfloat16>(o.planes * o.plane_step);
  return o;
}

// A matrix as the tensor cores take it: in place, or copied (the launches of a call follow it).
cudaError_t operand(const Source& m, bool f32, Room& room, bool launch, cudaStream_t s, MmOperand& o) {
  if (!f32 && reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && (m.rows <= 1 || (m.ld % 8 == 0 && m.ld >= m.inner)) &&
      (m.halves == 1 || (m.half_step % 8 == 0 && m.half_step > 0)) &&
      (m.experts == 1 || (m.expert_step % 8 == 0 && m.expert_step > 0))) {
    o.p = static_cast<const __nv_bfloat16*>(m.p);
    o.inner = m.inner, o.rows = m.rows, o.ld = m.ld, o.half_step = m.half_step, o.expert_step = m.expert_step;
    o.halves = m.halves, o.experts = m.experts;
    return cudaSuccess;
  }
  o = packed(room, m.inner, m.rows, m.halves, m.experts, f32);
  if (!launch) return cudaSuccess;
  PackArgs a;
  a.src = m.p, a.ld = m.ld, a.half_step = m.half_step, a.expert_step = m.expert_step;
  a.f32 = f32, a.last = m.last, a.to = o;
  return launch_expert_pack(a, s);
}

// Rows of a part of a weight gradient with M x N outputs, 0: no parts.  With fewer than two tiles for each
// pair of SMs, the rows are cut so that there are about three.
int split_rows(int64_t rows, int experts, int64_t M, int64_t N) {
  const int64_t each = ((M + 255) / 256) * ((N + 255) / 256), pairs = std::max(1, device_sms() / 2);
  if (experts * each >= 2 * pairs) return 0;
  const int64_t cut = std::max<int64_t>(512, (rows * each / (3 * pairs) + 63) / 64 * 64);
  return cut * experts < rows ? (int)cut : 0;
}

cudaError_t product(const emb_product& p, ProductKind kind, Room& room, bool launch, cudaStream_t s) {
  const bool f32 = p.dtype == EMB_F32, gated = kind == kGated || kind == kGatedBackward;
  const bool back = kind == kLinearBackward || kind == kGatedBackward;
  const int64_t S = p.rows, in = p.in, f = p.out, O = gated ? 2 * f : f;
  const int32_t* last = p.d_offsets ? p.d_offsets + p.experts : nullptr;
  cudaError_t e = cudaSuccess;
  MmArgs a;
  a.offsets = p.d_offsets, a.E = p.experts, a.S = (int)S, a.f32 = f32;
  const Source x{p.d_x, in, S, p.x_ld, 0, 0, 1, 1, last};
  if (!back) {
    if (S == 0) return cudaSuccess;
    Source w{p.d_w, p.w_turned ? f : in, p.w_turned ? in : f, p.w_ld, p.w_turned ? f : f * p.w_ld, p.w_step, gated ? 2 : 1, p.experts};
    if ((e = operand(x, f32, room, launch, s, a.a)) != cudaSuccess) return e;
    if ((e = operand(w, f32, room, launch, s, a.b)) != cudaSuccess || !launch) return e;
    a.b_mn = p.w_turned != 0;
    a.N = (int)f, a.K = (int)in, a.act = gated ? p.act : -1;
    a.out = p.d_out, a.out_ld = p.out_ld, a.out_bf16 = !f32;
    if (gated) a.gu = p.d_gu, a.gu_ld = p.gu_ld;
    return launch_expert_mm_rows(a, s);
  }
  MmOperand d;  // [dg, du], or dout
  if (S > 0) {
    if (gated) {
      d = packed(room, O, S, 1, 1, f32);
      if (launch) e = launch_expert_gated_bwd(p, d, s);
    } else {
      e = operand({p.d_dout, f, S, p.dout_ld, 0, 0, 1, 1, last}, f32, room, launch, s, d);
    }
    if (e != cudaSuccess) return e;
  }
  if (p.d_dx && S > 0) {
    a.a = d;
    const Source w{p.d_w, p.w_turned ? O : in, p.w_turned ? in : O, p.w_ld, 0, p.w_step, 1, p.experts};
    if ((e = operand(w, f32, room, launch, s, a.b)) != cudaSuccess) return e;
    a.b_mn = p.w_turned == 0;
    a.N = (int)in, a.K = (int)O;
    a.out = p.d_dx, a.out_ld = p.dx_ld, a.out_bf16 = !f32;
    if (launch && (e = launch_expert_mm_rows(a, s)) != cudaSuccess) return e;
  }
  if (p.d_dw) {
    MmOperand xo;
    if (S > 0 && (e = operand(x, f32, room, launch, s, xo)) != cudaSuccess) return e;
    a.a = p.dw_turned ? xo : d, a.b = p.dw_turned ? d : xo;
    a.M = (int)(p.dw_turned ? in : O), a.N = (int)(p.dw_turned ? O : in), a.K = 0;
    a.out = p.d_dw, a.out_ld = p.dw_ld, a.out_step = p.dw_step, a.out_bf16 = p.dw_dtype == EMB_BF16;
    a.split = split_rows(S, p.experts, a.M, a.N);
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
